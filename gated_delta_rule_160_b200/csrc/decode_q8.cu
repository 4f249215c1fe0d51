// decode_q8.cu -- decode on an 8-bit state pool (q8.cuh): n_tok new tokens per sequence, each
// state read as codes, advanced in fp32 and quantised as it is written.
//
// With g_i = alpha_i s_i (decay and the row's scale; the decay alone from the second token on, when
// the state is already in fp32), v the codes' values, e = b (.) k and x = w (.) v_t:
//   r_j = sum_i k_i g_i v_ij,  p_j = sum_i q_i g_i v_ij
//   S_ij = g_i v_ij + (k_i x_j - e_i r_j),   o_j = p_j - (q . e) r_j + (q . k) x_j
// so the codes are scaled once, where the new state is formed. Between the tokens of one call the
// state stays in fp32 registers; only what is written to the pool, or to the per-token states, is
// rounded.
//
// Persistent CTAs of 8 warps, two per SM, walk the (sequence, value head) items. One thread brings
// the items two ahead into a ring of stages by bulk copies (codes, scales and token rows are
// contiguous each), so HBM latency stays out of the way. Warp w owns key rows w DK / 8 ..; lane l
// holds DV / 32 neighbouring columns of them. A row then lies in one warp: its largest magnitude is
// one warp-wide reduction instruction, its factors are staged by the warp for itself, and its
// codes leave as one 64- or 128-byte store. The two column sums cross the warps through shared
// memory, which is the one barrier per token. Registers hold the state as pairs of rows: packed
// two-wide arithmetic then takes the rows' factors as they lie in shared memory.
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace {

// Device status word of this file's kernels (kStatus* bits), read and cleared by
// gdn2_device_status.
__device__ unsigned int g_status_q8 = 0;

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(mbar)
                 : "memory");
}

template <int N> struct Word;  // the codes of N neighbouring columns
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<4> { using type = uint32_t; };

template <typename T, int N> struct alignas(sizeof(T) * N) Cols { T x[N]; };  // neighbouring columns, as one access

__device__ __forceinline__ float amax_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}
__device__ __forceinline__ float amax_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return d;
}

// One stage of the ring: codes, scales, and n_tok records [k, q, b, log_alpha or a, v, w].
struct StageLayout {
    int es, rec, rk, rq, rb, ra, rv, rw, bytes;
    __host__ __device__ StageLayout(int dk, int dv, bool bf16, bool pro, int n_tok) {
        es = bf16 ? 2 : 4;
        rk = 0;
        rq = dk * es;
        rb = 2 * dk * es;
        ra = 3 * dk * es;
        rv = ra + dk * (pro ? es : 4);
        rw = rv + dv * es;
        rec = rw + dv * es;
        bytes = dk * dv + dk * 4 + n_tok * rec;
    }
};

struct Ring {
    int stages, stage_bytes;
};

template <int DK, int DV, int kFmt, typename T, bool kPro>
__global__ void __launch_bounds__(kThreads, 2) decode_q8_kernel(const __grid_constant__ Params p, const __grid_constant__ Q8Args a,
                                                                const Ring ring) {
    constexpr int RW = DK / kWarps, CPL = DV / 32;  // rows per warp, columns per lane
    constexpr int kMaxStages = 3;
    using W = typename Word<CPL>::type;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ __align__(16) float red[2][2][kWarps][DV];  // [token parity][r | p][warp][column]
    __shared__ __align__(16) float dsum[2][kWarps][4];     // q . e, q . k, |q|^2, |k|^2 of a warp's rows
    __shared__ __align__(16) float rows[kWarps][6][RW];  // k g, q g, g, k, -e; row maxima, then 1 / scale
    __shared__ __align__(16) int4 head[kMaxStages];      // item (-1: no more), n, h, slot written
    __shared__ __align__(8) uint64_t full[kMaxStages];

    const StageLayout L(DK, DV, sizeof(T) == 2, kPro, p.n_tok);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, n_tok = p.n_tok;
    const int n_items = p.n_seq * p.h_v;
    const uint32_t full0 = tc::smem_u32(full), dsm0 = tc::smem_u32(dsm);

    // ---- producer (thread 0): the next active item and its slots are known one issue ahead
    int nit = blockIdx.x, nslot = -1, nout = -1, issued = 0;
    bool ended = false;
    auto look = [&]() {
        for (; nit < n_items; nit += gridDim.x) {
            const int n = nit / p.h_v;
            nslot = p.slots ? p.slots[n] : n;
            if (nslot >= 0 && nslot < p.n_slots) {
                nout = a.slots_out ? a.slots_out[n] : nslot;
                break;
            }
        }
    };
    auto issue = [&]() {
        if (ended) return;
        const int s = issued % ring.stages;
        const uint32_t bar = full0 + 8 * s, dst = dsm0 + s * ring.stage_bytes;
        ++issued;
        if (nit >= n_items) {
            ended = true;
            head[s] = make_int4(-1, 0, 0, 0);
            tc::mbar_arrive(bar);
            return;
        }
        const int n = nit / p.h_v, h = nit % p.h_v, g = h / (p.h_v / p.h_qk);
        head[s] = make_int4(nit, n, h, nout);
        tc::mbar_expect_tx(bar, L.bytes);
        const size_t st = (size_t)nslot * p.h_v + h;
        bulk_load(dst, static_cast<const uint8_t*>(a.codes) + st * (DK * DV), DK * DV, bar);
        bulk_load(dst + DK * DV, a.scales + st * DK, DK * 4, bar);
        for (int t = 0; t < n_tok; ++t) {
            const uint32_t rec = dst + DK * DV + DK * 4 + t * L.rec;
            const size_t row = (size_t)n * n_tok + t, tq = (row * p.h_qk + g) * DK, tk = (row * p.h_v + h) * DK, tv = (row * p.h_v + h) * DV;
            bulk_load(rec + L.rk, static_cast<const T*>(p.k) + tq, DK * sizeof(T), bar);
            bulk_load(rec + L.rq, static_cast<const T*>(p.q) + tq, DK * sizeof(T), bar);
            bulk_load(rec + L.rb, static_cast<const T*>(p.b) + tk, DK * sizeof(T), bar);
            if (kPro)
                bulk_load(rec + L.ra, static_cast<const T*>(p.a_raw) + tk, DK * sizeof(T), bar);
            else
                bulk_load(rec + L.ra, p.log_alpha + tk, DK * 4, bar);
            bulk_load(rec + L.rv, static_cast<const T*>(p.v) + tv, DV * sizeof(T), bar);
            bulk_load(rec + L.rw, static_cast<const T*>(p.w) + tv, DV * sizeof(T), bar);
        }
        nit += gridDim.x;
        look();
    };

    if (tid == 0) {
        for (int s = 0; s < ring.stages; ++s) tc::mbar_init(full0 + 8 * s, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    if (tid == 0 && !p.test_withhold_loads) {
        look();
        for (int s = 0; s + 1 < ring.stages; ++s) issue();
    }

    float(*rv)[RW] = rows[warp];
    const int c0 = lane * CPL;
    int buf = 0, st = 0;
    uint32_t parity = 0;
    bool fault = false;
    int taken = 0;  // stages waited for
    for (;; ++taken, st = st + 1 == ring.stages ? (parity ^= 1u, 0) : st + 1) {
        // bounded: a load that never lands ends the kernel with a status bit, not a hang
        if (!tc::mbar_wait(full0 + 8 * st, parity, p.wait_ns)) fault = true;
        const int4 hd = fault ? make_int4(0, 0, 0, -1) : head[st];
        if (hd.x < 0) break;
        const uint8_t* stage = dsm + st * ring.stage_bytes;
        const float* scales = reinterpret_cast<const float*>(stage + DK * DV);
        const uint8_t* rec = stage + DK * DV + DK * 4;

        // this lane's columns of the warp's rows, as values of the codes, in pairs of rows
        float2 v[RW / 2][CPL];
#pragma unroll
        for (int i = 0; i < RW / 2; ++i) {
            const uint8_t* at = stage + (size_t)(warp * RW + 2 * i) * DV + c0;
            q8_unpack_pair<kFmt, CPL>(*reinterpret_cast<const W*>(at), *reinterpret_cast<const W*>(at + DV), v[i]);
        }
        for (int t = 0; t < n_tok; ++t, rec += L.rec, buf ^= 1) {
            // the warp's row factors
            __syncwarp();
            float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
            if (lane < RW) {
                const int i = warp * RW + lane;
                const float kv = to_f32(reinterpret_cast<const T*>(rec + L.rk)[i]), qv = to_f32(reinterpret_cast<const T*>(rec + L.rq)[i]);
                float bv = to_f32(reinterpret_cast<const T*>(rec + L.rb)[i]);
                float g;
                if (kPro) {
                    g = sigmoid_f(-to_f32(reinterpret_cast<const T*>(rec + L.ra)[i]));
                    bv = sigmoid_f(bv);
                } else {
                    g = expf(reinterpret_cast<const float*>(rec + L.ra)[i]);
                }
                if (t == 0) g *= scales[i];
                const float e = bv * kv;
                rv[0][lane] = kv * g;
                rv[1][lane] = qv * g;
                rv[2][lane] = g;
                rv[3][lane] = kv;
                rv[4][lane] = -e;
                d0 = qv * e;
                d1 = qv * kv;
                if (kPro) {
                    d2 = qv * qv;
                    d3 = kv * kv;
                }
            }
#pragma unroll
            for (int off = RW / 2; off > 0; off >>= 1) {
                d0 += __shfl_xor_sync(0xffffffffu, d0, off);
                d1 += __shfl_xor_sync(0xffffffffu, d1, off);
                if (kPro) {
                    d2 += __shfl_xor_sync(0xffffffffu, d2, off);
                    d3 += __shfl_xor_sync(0xffffffffu, d3, off);
                }
            }
            if (lane == 0) *reinterpret_cast<float4*>(dsum[buf][warp]) = make_float4(d0, d1, d2, d3);
            __syncwarp();

            float2 r2[CPL], p2[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) r2[j] = p2[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {
                const float4 kg = *reinterpret_cast<const float4*>(&rv[0][4 * i]), qg = *reinterpret_cast<const float4*>(&rv[1][4 * i]);
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    r2[j] = ffma2(make_float2(kg.x, kg.y), v[2 * i][j], r2[j]);
                    p2[j] = ffma2(make_float2(qg.x, qg.y), v[2 * i][j], p2[j]);
                    r2[j] = ffma2(make_float2(kg.z, kg.w), v[2 * i + 1][j], r2[j]);
                    p2[j] = ffma2(make_float2(qg.z, qg.w), v[2 * i + 1][j], p2[j]);
                }
            }
            Cols<float, CPL> rs, ps;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                rs.x[j] = r2[j].x + r2[j].y;
                ps.x[j] = p2[j].x + p2[j].y;
            }
            *reinterpret_cast<Cols<float, CPL>*>(&red[buf][0][warp][c0]) = rs;
            *reinterpret_cast<Cols<float, CPL>*>(&red[buf][1][warp][c0]) = ps;
            // every warp's sums are in; every warp is done with the previous item, too
            if (__syncthreads_or(fault)) {
                fault = true;
                break;
            }
            if (t == 0 && tid == 0) issue();
            float r[CPL];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const Cols<float, CPL> y = *reinterpret_cast<const Cols<float, CPL>*>(&red[buf][0][w][c0]);
#pragma unroll
                for (int j = 0; j < CPL; ++j) r[j] = w == 0 ? y.x[j] : r[j] + y.x[j];
            }
            // fused pre-processing: q and k enter unnormalised, and each sum takes its norms here
            float nq = 1.f, nk = 1.f;
            if (kPro) {
                float sq = 0.f, sk = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    sq += dsum[buf][w][2];
                    sk += dsum[buf][w][3];
                }
                nq = 1.f / fmaxf(sqrtf(sq), kL2NormEps);
                nk = 1.f / fmaxf(sqrtf(sk), kL2NormEps);
            }
            const T *tv = reinterpret_cast<const T*>(rec + L.rv), *tw = reinterpret_cast<const T*>(rec + L.rw);
            auto write = [](T w, T v_t) { return (kPro ? sigmoid_f(to_f32(w)) : to_f32(w)) * to_f32(v_t); };  // x = w (.) v
            const size_t row = ((size_t)hd.y * n_tok + t) * p.h_v + hd.z;
            if (tid < DV) {
                float pj = 0.f, rj = 0.f, qe = 0.f, qk = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    rj += red[buf][0][w][tid];
                    pj += red[buf][1][w][tid];
                    qe += dsum[buf][w][0];
                    qk += dsum[buf][w][1];
                }
                const float o = nq * (pj + nk * (qk * write(tw[tid], tv[tid]) - qe * (nk * rj)));
                if (a.o_bf16)
                    static_cast<__nv_bfloat16*>(p.o)[row * DV + tid] = __float2bfloat16_rn(o);
                else
                    static_cast<float*>(p.o)[row * DV + tid] = o;
            }
            float x[CPL];
            const Cols<T, CPL> wc = *reinterpret_cast<const Cols<T, CPL>*>(tw + c0), vc = *reinterpret_cast<const Cols<T, CPL>*>(tv + c0);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                x[j] = nk * write(wc.x[j], vc.x[j]);
                r[j] *= nk * nk;
            }
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {
                const float4 g4 = *reinterpret_cast<const float4*>(&rv[2][4 * i]), k4 = *reinterpret_cast<const float4*>(&rv[3][4 * i]);
                const float4 e4 = *reinterpret_cast<const float4*>(&rv[4][4 * i]);
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    v[2 * i][j] = ffma2(make_float2(g4.x, g4.y), v[2 * i][j],
                                        ffma2(make_float2(k4.x, k4.y), dup2(x[j]), fmul2(make_float2(e4.x, e4.y), dup2(r[j]))));
                    v[2 * i + 1][j] = ffma2(make_float2(g4.z, g4.w), v[2 * i + 1][j],
                                            ffma2(make_float2(k4.z, k4.w), dup2(x[j]), fmul2(make_float2(e4.z, e4.w), dup2(r[j]))));
                }
            }
            const bool last = t + 1 == n_tok;
            if (!last && !a.code_steps) continue;

            // quantise: the row maxima, then one row's scale per lane
            float m[RW];
#pragma unroll
            for (int i = 0; i < RW / 2; ++i) {
                if (CPL == 4) {
                    m[2 * i] = amax_nan(amax_nan(v[i][0].x, v[i][1].x, v[i][2 % CPL].x), v[i][3 % CPL].x);
                    m[2 * i + 1] = amax_nan(amax_nan(v[i][0].y, v[i][1].y, v[i][2 % CPL].y), v[i][3 % CPL].y);
                } else {
                    m[2 * i] = amax_nan(v[i][0].x, v[i][1].x);
                    m[2 * i + 1] = amax_nan(v[i][0].y, v[i][1].y);
                }
            }
#pragma unroll
            for (int i = 0; i < RW; ++i) m[i] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[i])));
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < RW / 4; ++i) *reinterpret_cast<float4*>(&rv[5][4 * i]) = make_float4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
            }
            __syncwarp();
            float scale = 0.f, inv = 1.f;
            if (lane < RW) {
                q8_scale<kFmt>(rv[5][lane], scale, inv);
                rv[5][lane] = inv;
            }
            __syncwarp();
            const bool zero_rows = __any_sync(0xffffffffu, inv == 0.f);
            uint32_t word[RW];
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {
                const float4 i4 = *reinterpret_cast<const float4*>(&rv[5][4 * i]);
                q8_pack_pair<kFmt, CPL>(v[2 * i], make_float2(i4.x, i4.y), word[4 * i], word[4 * i + 1]);
                q8_pack_pair<kFmt, CPL>(v[2 * i + 1], make_float2(i4.z, i4.w), word[4 * i + 2], word[4 * i + 3]);
            }
            if (zero_rows) {  // rows whose codes are 0 whatever they hold
#pragma unroll
                for (int i = 0; i < RW; ++i) word[i] = rv[5][i] == 0.f ? 0u : word[i];
            }
            auto put = [&](void* codes, float* sc, size_t state) {
                uint8_t* at = static_cast<uint8_t*>(codes) + state * (DK * DV) + (size_t)warp * RW * DV + c0;
#pragma unroll
                for (int i = 0; i < RW; ++i) *reinterpret_cast<W*>(at + i * DV) = (W)word[i];
                if (lane < RW) sc[state * DK + warp * RW + lane] = scale;
            };
            if (a.code_steps) put(a.code_steps, a.scale_steps, row);
            if (last && hd.w >= 0 && hd.w < p.n_slots) put(a.codes, a.scales, (size_t)hd.w * p.h_v + hd.z);
        }
        if (fault) break;
    }
    if (fault && tid == 0) {
        atomicOr(&g_status_q8, kStatusWaitTimeout);
        // give loads still in flight a last bounded chance to land before the CTA exits
        for (int i = taken; i < issued; ++i) tc::mbar_wait(full0 + 8 * (i % ring.stages), (i / ring.stages) & 1, p.wait_ns);
    }
}

template <int DK, int DV, int kFmt, typename T, bool kPro>
cudaError_t launch(const Params& p, const Q8Args& a, cudaStream_t st) {
    auto kern = decode_q8_kernel<DK, DV, kFmt, T, kPro>;
    const StageLayout L(DK, DV, sizeof(T) == 2, kPro, p.n_tok);
    Ring ring;
    ring.stage_bytes = (L.bytes + 127) & ~127;
    // three stages (two items ahead) where two CTAs of them fit an SM, else two
    ring.stages = 3 * ring.stage_bytes <= 90 * 1024 ? 3 : 2;
    const int smem = ring.stages * ring.stage_bytes;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int items = p.n_seq * p.h_v;
    kern<<<items < sms * per_sm ? items : sms * per_sm, kThreads, smem, st>>>(p, a, ring);
    return cudaGetLastError();
}

template <int DK, int DV, int kFmt>
cudaError_t launch_t(const Params& p, const Q8Args& a, cudaStream_t st) {
    if (a.bf16) return p.prologue ? launch<DK, DV, kFmt, __nv_bfloat16, true>(p, a, st) : launch<DK, DV, kFmt, __nv_bfloat16, false>(p, a, st);
    return p.prologue ? launch<DK, DV, kFmt, float, true>(p, a, st) : launch<DK, DV, kFmt, float, false>(p, a, st);
}

template <int kFmt>
cudaError_t launch_f(const Params& p, const Q8Args& a, cudaStream_t st) {
    if (p.dk == 128) return p.dv == 128 ? launch_t<128, 128, kFmt>(p, a, st) : launch_t<128, 64, kFmt>(p, a, st);
    return p.dv == 128 ? launch_t<64, 128, kFmt>(p, a, st) : launch_t<64, 64, kFmt>(p, a, st);
}

}  // namespace

cudaError_t read_clear_status_decode_q8(unsigned int* out, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_status_q8, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, s);
    if (e != cudaSuccess) return e;
    static const unsigned int zero = 0;
    return cudaMemcpyToSymbolAsync(g_status_q8, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, s);
}

cudaError_t launch_decode_q8(const Params& p, const Q8Args& a, cudaStream_t st) {
    return a.fmt == GDN2_Q8_INT8 ? launch_f<GDN2_Q8_INT8>(p, a, st) : launch_f<GDN2_Q8_E4M3>(p, a, st);
}

}  // namespace gdn2
