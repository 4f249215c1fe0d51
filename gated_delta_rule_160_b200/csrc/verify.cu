// verify.cu -- verification of drafted tokens against the target's probabilities, from given
// random numbers (gdn2_verify_drafts).
//
// Of sequence n's drafted tokens t_0 .. t_{m-1}, token i is accepted while u_i q_i(t_i) < p_i(t_i).
// The first one that is not is replaced by a token of the residual r = max(p_i - q_i, 0) (of p_i
// where r is empty); with all accepted one more token comes from p_m. Tokens are drawn by inverse
// CDF: the lowest j with r_0 + .. + r_j > u (r_0 + .. + r_{V-1}).
//
// Acceptance is decided in fp64 from the exact values of the inputs (u q is exact there: 24 + 24 bits).
// A difference p - q is rounded to fp32 and added in fp64; what the rounding took off, at most 2^-24 of
// it, is exact in fp32, is added there as a tree over 16 values (four roundings: 2^-46 of the weights)
// and then in fp64. With the 100 fp64 additions at most on a value's way to the border (100 2^-53),
// sums are good to 2^-45 of the weights in them; over 131072 tokens the order of the additions then
// shows in at most one draw of 10^7. (256 rows of 131072 fp32 values: 48.5 us; the trees over 4 values
// only 50.5; both operands converted to fp64 61; remainders added one by one over a segment 48.4, but
// good to 2^-43 only.)
//
// The work is one row of p and, where a draft was refused, one of q a sequence. A cluster of up to 8
// CTAs shares a sequence: each warp sums segments of 1024 weights with half a segment in flight, the
// CTAs exchange their sums through distributed shared memory, and the CTA that holds the border scans
// its segment sums and then that one segment again, out of L2. No workspace, no atomics on memory, one
// launch. Measured on B200, 256 sequences, 4 drafts, 131072 values a row, 1.87 rows read a sequence:
// fp32 48.4 us, 0.80 of the copy bandwidth, bound by HBM and by the accept phase of each cluster; bf16
// 36.0 us, 0.54: half the bytes, but as many instructions (10.5 M warp instructions for 128 rows, 10.8
// M in fp32: a minimum, three subtractions, two additions and a conversion a value). They take 18 us of
// the 36 at full rate; 55 % of issue slots are used, and what waits waits for loads. Certain drafts,
// which read p alone: 38.9 us in fp32 (0.53), 36.3 in bf16 (0.29). Rows that do not start at 16-byte
// boundaries: 56.5 and 62.9 us. One sequence, 3 drafts, 32768 values: 6.5 us, the latency of drafts,
// their probabilities, the row and its segment again, one after the other.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.cuh"

namespace cg = cooperative_groups;

namespace gdn2 {
namespace {

constexpr int kSeg = 1024;         // values per segment of the CDF; a warp sums one at a time
constexpr int kMaxCluster = 8;     // CTAs per sequence (the portable cluster size)
constexpr int kMaxSeg = GDN2_VERIFY_MAX_VOCAB / kSeg / kMaxCluster;  // segments per CTA

enum Mode { kPlain, kResidual, kOneHot };

// A probability as it counts: positive and finite, else 0 (as integers, everything else is larger).
__device__ __forceinline__ float clean(float x) { return __float_as_uint(x) < 0x7f800000u ? x : 0.f; }

// 16 bytes of probabilities as floats.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void get(uint4 v, float* x) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void get(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// The weight of a token in the row that the next token is drawn from.
__device__ __forceinline__ double weight(float p, float q, bool masked) {
    p = clean(p);
    q = clean(q);
    return p > q && !masked ? (double)p - (double)q : 0.0;
}

template <typename T>
struct Row {
    const T* p;
    const T* q;  // kResidual
    int t;       // kOneHot: the token left out
    int mode;
    __device__ __forceinline__ double at(int j) const {
        return weight(to_f32(p[j]), mode == kResidual ? to_f32(q[j]) : 0.f, mode == kOneHot && j == t);
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

// The sum of N values as a balanced tree: log2 N roundings on each.
template <int N>
__device__ __forceinline__ float tree_sum(const float* x) {
    if constexpr (N == 1) return x[0];
    else return tree_sum<N / 2>(x) + tree_sum<N / 2>(x + N / 2);
}

// Add the weights of the N tokens j, j + kStep, .. to s and return the sum of what the differences among
// them rounded off; nearly all rows hold only finite values from 0 up, which one comparison finds out for
// all N.
template <int N, int kStep = 1>
__device__ __forceinline__ float add(double& s, float* p, float* q, int mode, int j, int t) {
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) most = max(most, __float_as_uint(p[e]));
    if (mode == kResidual) {
#pragma unroll
        for (int e = 0; e < N; ++e) most = max(most, __float_as_uint(q[e]));
    }
    if (most >= 0x7f800000u) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            p[e] = clean(p[e]);
            q[e] = clean(q[e]);
        }
    }
    if (mode != kResidual) {
#pragma unroll
        for (int e = 0; e < N; ++e) s += (double)(mode == kOneHot && j + e * kStep == t ? 0.f : p[e]);
        return 0.f;
    }
    float lost[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float m = fminf(p[e], q[e]);         // p - m = max(p - q, 0)
        const float d = __fsub_rn(p[e], m);
        lost[e] = __fsub_rn(__fsub_rn(p[e], d), m);  // what d rounded off (p >= m >= 0: exact)
        s += (double)d;
    }
    return tree_sum<N>(lost);
}

// 16 bytes at `at`, wherever the row (lo up to hi) starts: the two 16-byte blocks around them, shifted. A
// block that reaches over an end of the row is put together value by value; bytes behind the row
// are 0. (Value by value, 48 odd rows of 50257 bf16 values took 14.0 us instead of 10.3; for 4-byte values
// the shifts cost more than they save.)
template <typename T>
__device__ __forceinline__ uint4 block(const char* at, const char* lo, const char* hi) {
    if (at >= lo && at + 16 <= hi) return __ldg(reinterpret_cast<const uint4*>(at));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; i += (int)sizeof(T)) {
        if (at + i >= lo && at + i < hi) {
            if (sizeof(T) == 4) w[i / 4] = *reinterpret_cast<const uint32_t*>(at + i);
            else w[i / 4] |= (uint32_t)*reinterpret_cast<const uint16_t*>(at + i) << (8 * (i % 4));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 load16(const T* x, const T* row, int V) {
    const char *at = reinterpret_cast<const char*>(x), *lo = reinterpret_cast<const char*>(row), *hi = reinterpret_cast<const char*>(row + V);
    const int s = (int)(reinterpret_cast<uintptr_t>(at) & 15);
    const uint4 a = block<T>(at - s, lo, hi);
    if (s == 0) return a;
    const uint4 b = block<T>(at - s + 16, lo, hi);
    uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    const uint32_t last = b.w;
    uint32_t u[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {  // from word s / 4 on
        const uint32_t w4 = i + 3 < 7 ? w[i + 3 < 7 ? i + 3 : 0] : last;
        const uint32_t even = s & 8 ? (i + 2 < 7 ? w[i + 2 < 7 ? i + 2 : 0] : last) : w[i], odd = s & 8 ? w4 : w[i + 1];
        u[i] = s & 4 ? odd : even;
    }
    const int bits = 8 * (s & 3);
    return make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits), __funnelshift_r(u[2], u[3], bits),
                      __funnelshift_r(u[3], u[4], bits));
}

// This lane's share of one segment's sum (streaming loads: 47.9 us, 49.1 without), kSeg / 2 (values of 4 bytes) or more loaded before their first
// use. Rows that start at 16-byte boundaries and hold whole vectors are read as such; others value by
// value in 4 bytes, as shifted vectors in 2.
template <typename T, bool kVec>
__device__ __forceinline__ double segment(const Row<T>& row, int j0, int V, int lane) {
    double s = 0.0;
    if (kVec || sizeof(T) == 2) {
        constexpr int N = Vec<T>::kN, IT = kSeg / (32 * N) / 2;
#pragma unroll 1
        for (int j1 = j0 + lane * N; j1 < j0 + kSeg; j1 += IT * 32 * N) {
            uint4 pv[IT], qv[IT];
            float lost[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int j = j1 + i * 32 * N;
                pv[i] = qv[i] = make_uint4(0, 0, 0, 0);
                if (j < V) {
                    pv[i] = kVec ? __ldcs(reinterpret_cast<const uint4*>(row.p + j)) : load16(row.p + j, row.p, V);
                    if (row.mode == kResidual) qv[i] = kVec ? __ldcs(reinterpret_cast<const uint4*>(row.q + j)) : load16(row.q + j, row.q, V);
                }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                float pf[N], qf[N];
                Vec<T>::get(pv[i], pf);
                Vec<T>::get(qv[i], qf);
                lost[i] = add<N>(s, pf, qf, row.mode, j1 + i * 32 * N, row.t);
            }
            if (row.mode == kResidual) s += (double)tree_sum<IT>(lost);
        }
    } else {
        constexpr int U = 16;
#pragma unroll 1
        for (int j1 = j0 + lane; j1 < j0 + kSeg; j1 += U * 32) {
            float pf[U], qf[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int j = j1 + i * 32;
                pf[i] = j < V ? to_f32(row.p[j]) : 0.f;
                qf[i] = j < V && row.mode == kResidual ? to_f32(row.q[j]) : 0.f;
            }
            const float lost = add<U, 32>(s, pf, qf, row.mode, j1, row.t);
            if (row.mode == kResidual) s += (double)lost;
        }
    }
    return s;
}

template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ double seg_sum[kMaxSeg];
    __shared__ double wsum[kWarps];
    __shared__ double cta_total[2];  // this CTA's part of the row, read by the whole cluster
    __shared__ double s_before;
    __shared__ int s_taken, s_seg, s_found, s_last;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int n = blockIdx.x / ctas, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int V = a.vocab, k = a.n_draft;
    int m = a.n_drafted ? a.n_drafted[n] : k;
    int* tokens = a.tokens + (size_t)n * (k + 1);
    if (m < 0) {  // an inactive sequence
        if (rank == 0 && tid <= k) tokens[tid] = -1;
        if (rank == 0 && tid == 0) a.n_accepted[n] = -1;
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
                const float pt = clean(to_f32(P[(size_t)lane * V + t])), qt = Q ? clean(to_f32(Q[(size_t)lane * V + t])) : 1.f;
                const float u = a.u_accept[(size_t)n * k + lane];
                // below 0 as 0 (else a token without target probability would pass); a NaN stays one and refuses
                yes = (u < 0.f ? 0.0 : (double)u) * (double)qt < (double)pt;
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

    // this CTA's segments, and their sum
    const int segs = (V + kSeg - 1) / kSeg, per = (segs + ctas - 1) / ctas;
    const int first = min(rank * per, segs), count = min(per, segs - first);
    double part[kMaxCluster], total = 0.0;
    for (int pass = 0;; ++pass) {
        for (int s = warp; s < count; s += kWarps) {
            const double x = warp_sum(segment<T, kVec>(row, (first + s) * kSeg, V, lane));
            if (lane == 0) seg_sum[s] = x;
        }
        __syncthreads();
        if (warp == 0) {
            double x = 0.0;
            for (int s = lane; s < count; s += 32) x += seg_sum[s];
            x = warp_sum(x);
            if (lane == 0) cta_total[pass] = x;
        }
        cluster.sync();
        total = 0.0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            part[c] = c < ctas ? *cluster.map_shared_rank(&cta_total[pass], c) : 0.0;
            total += part[c];
        }
        if (total > 0.0 || row.mode == kPlain) break;
        row.mode = kPlain;  // nothing is left of the row: its own probabilities
    }
    cluster.barrier_arrive();  // no more reads of other CTAs' shared memory
    // Every CTA has the same sums, so all agree on the one that holds the border: the first whose
    // running sum passes the target, else (a random number of 1, a rounding) the last with any weight.
    const double target = fmin(fmax((double)a.u_sample[n], 0.0), 1.0) * total;
    int owner = 0;
    double run = 0.0, before = 0.0;
    bool found_cta = false;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
        if (part[c] > 0.0 && !found_cta) {
            owner = c;
            before = run;
            found_cta = run + part[c] > target;
        }
        run += part[c];
    }
    if (rank == owner) {
        int token = -1;
        if (total > 0.0) {
            // the segment, by the same rule
            if (warp == 0) {
                double run = before, at = 0.0, last_at = 0.0;
                int found = -1, last = -1;
                for (int s0 = 0; s0 < count && found < 0; s0 += 32) {
                    const double x = s0 + lane < count ? seg_sum[s0 + lane] : 0.0;
                    const double c = run + warp_scan(x, lane);
                    const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
                    const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && c > target);
                    if (hit) {
                        const int l = __ffs(hit) - 1;
                        found = s0 + l;
                        at = __shfl_sync(0xffffffffu, c - x, l);
                    } else if (some) {
                        const int l = 31 - __clz(some);
                        last = s0 + l;
                        last_at = __shfl_sync(0xffffffffu, c - x, l);
                    }
                    run = __shfl_sync(0xffffffffu, c, 31);
                }
                if (lane == 0) {
                    s_seg = found >= 0 ? found : last;
                    s_before = found >= 0 ? at : last_at;
                    s_found = 0x7fffffff;
                    s_last = -1;
                }
            }
            __syncthreads();
            // the token within the segment
            constexpr int E = kSeg / kThreads;
            const int j0 = (first + s_seg) * kSeg + tid * E;
            double x[E], sum = 0.0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                x[i] = j0 + i < V ? row.at(j0 + i) : 0.0;
                sum += x[i];
            }
            const double c = warp_scan(sum, lane);
            if (lane == 31) wsum[warp] = c;
            __syncthreads();
            double run = s_before + (c - sum);
            for (int w = 0; w < warp; ++w) run += wsum[w];
            int found = 0x7fffffff, last = -1;
#pragma unroll
            for (int i = 0; i < E; ++i) {
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
        if (tid <= k) tokens[tid] = tid < taken ? drafts[tid] : (tid == taken ? token : -1);
        if (tid == 0) a.n_accepted[n] = taken;
    }
    cluster.barrier_wait();  // this CTA's sums stay readable until all have read them
}

template <typename T, bool kVec, int kThreads>
cudaError_t launch(const VerifyArgs& a, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.n_seq * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, kVec, kThreads>, a);
}

template <typename T, bool kVec>
cudaError_t launch_v(const VerifyArgs& a, cudaStream_t st) {
    // CTAs of 4 warps for large batches, of 8 for small ones; in the cluster one segment for each warp, as far
    // as 8 CTAs go. 74 clusters of 8 x 8 warps are resident at a time, and up to there more warps a
    // sequence win: 64 rows of 131072 values 15.1 us against 17.7 (fp32) and 13.5 against 15.6 (bf16). Beyond, the
    // shorter CTAs overlap one sequence's loads with another's exchange: 128 rows 24.9 against 27.3 and 20.2
    // against 23.5, 256 rows 45.0 against 49.1 and 36.2 against 43.1. With 32768 values or fewer the two are
    // within 5 % of each other. The rule changes over at 128 rows (32 segments or more); 96 rows, on
    // the 8-warp side, take 23.9 us where the other takes 21.4.
    const int segs = (a.vocab + kSeg - 1) / kSeg;
    const bool full = (long long)a.n_seq * std::min(segs, kMaxCluster * 4) >= 4096;
    int ctas = 1;
    while (ctas < kMaxCluster && ctas * (full ? 4 : 8) < segs) ctas *= 2;
    return full ? launch<T, kVec, 128>(a, ctas, st) : launch<T, kVec, 256>(a, ctas, st);
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t st) {
    const auto whole = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; };
    return whole(a.p) && whole(a.q) && a.vocab % Vec<T>::kN == 0 ? launch_v<T, true>(a, st) : launch_v<T, false>(a, st);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, gdn2_dtype dt, cudaStream_t st) {
    return dt == GDN2_F32 ? launch_t<float>(a, st) : launch_t<__nv_bfloat16>(a, st);
}

}  // namespace gdn2
