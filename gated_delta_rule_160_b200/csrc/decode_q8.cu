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
// Persistent CTAs walk the (sequence, value head) items. The next items come into a ring of stages
// by bulk copies (codes, scales and token rows are contiguous each), so HBM latency stays out of the
// way. Warp w owns key rows w DK / W ..; lane l holds DV / 32 neighbouring columns of them. A row
// then lies in one warp: its largest magnitude is one warp-wide reduction instruction, its factors
// are staged by the warp for itself, and its codes leave as one 64- or 128-byte store. The two
// column sums cross the warps through shared memory, which is the one barrier per token. The
// arithmetic runs on pairs of rows: packed two-wide instructions take the rows' factors as they
// lie in shared memory.
//
// Measured on B200, 256 sequences x 32 heads x 128 x 128, e4m3, one token: 80.3 us for 0.296 GB of
// codes, scales and tokens (3.68 TB/s, 0.57 of the copy bandwidth; the fp32 pool takes 165 us). int8
// 81.0, from raw projections 84.0 and 84.2. Neither HBM nor the issue of instructions bounds it: the
// 5.6 K warp instructions of an item would take half of that at full rate, and 9 % fewer of them were
// no faster. It is latency. An item is one chain of factors, sums, barrier, update, magnitudes, scales
// and rounding; 4 warps a scheduler fill 52 % of its issue slots, the first stall is the barrier, and
// more warps per SM (fewer registers each) did not help. 64 sequences, 4 tokens: with the state after
// each 83.4 us (floor 35.1; int8 84.5, raw 93.9), without 64.5 (floor 13.6; int8 65.6, raw 75.9), by
// the same chain a token. The 128 x 128 forms for several raw tokens spill 8 to 16 bytes at 128
// registers.
#include <algorithm>
#include <atomic>

#include "q8.cuh"
#include "tc_ptx.cuh"

namespace gdn2 {
namespace {

// Device status word of this file's kernels (kStatus* bits), read and cleared by
// gdn2_device_status.
__device__ unsigned int g_status_q8 = 0;

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

// Four neighbouring floats of shared memory as two pairs.
__device__ __forceinline__ ulonglong2 pairs(const float* x) { return *reinterpret_cast<const ulonglong2*>(x); }

// This lane's columns summed over the warps, as pairs of columns: partial sums of DK / 8 rows each, in
// pairs first. With 4 warps the pairs have been added already, so both forms of the kernel
// give the same bits.
template <int CPL, int W, int DV>
__device__ __forceinline__ void sum_warps(const float (&x)[W][DV], int c0, f32x2* s) {
#pragma unroll
    for (int w = 0; w < W; w += W / 4) {
#pragma unroll
        for (int j = 0; j < CPL / 2; ++j) {
            f32x2 y = *reinterpret_cast<const f32x2*>(&x[w][c0 + 2 * j]);
            if (W == 8) y = add2(y, *reinterpret_cast<const f32x2*>(&x[(w + 1) % W][c0 + 2 * j]));
            s[j] = w == 0 ? y : add2(s[j], y);
        }
    }
}
template <int W>
__device__ __forceinline__ float sum_dots(const float (&x)[W][4], int c) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; w += W / 4) {
        const float y = W == 8 ? x[w][c] + x[(w + 1) % W][c] : x[w][c];
        s = w == 0 ? y : s + y;
    }
    return s;
}

struct Ring {
    int stages, stage_bytes;
    const void* src[8];  // what a stage is brought from: codes, scales, k, q, b, log_alpha or a, v, w
};

// kOne: one token and no per-token states. 4 CTAs of 4 warps then fit an SM, and the work that a
// warp does once per token is spread over twice the rows: a thread keeps the values of one half of its
// rows from the sums to the update, and reads the other half's codes again (85.5 us with 4 CTAs of
// 4 warps that read all of them again, 101.6 us with 2 of 8 that keep all). Otherwise 2 CTAs of 8
// warps, the state in registers from token to token.
template <int DK, int DV, int kFmt, typename T, bool kPro, bool kOne>
struct Cfg {
    static constexpr int W = kOne ? 4 : 8, NT = 32 * W, CTAS = kOne ? 4 : 2;
    static constexpr int RW = DK / W, CPL = DV / 32;       // rows per warp, columns per lane
    static constexpr int G = RW < 16 ? RW : 16;            // rows quantised at a time
    static constexpr int ES = sizeof(T), AB = kPro ? DK * ES : DK * 4;
    static constexpr int RK = 0, RQ = DK * ES, RB = 2 * DK * ES, RA = 3 * DK * ES, RV = RA + AB, RWR = RV + DV * ES;
    static constexpr int REC = RWR + DV * ES;              // one token's record in a stage
    static constexpr int TOK = DK * DV + DK * 4;           // where the records start
    static constexpr int MAX_STAGES = 3;
};

template <int DK, int DV, int kFmt, typename T, bool kPro, bool kOne>
__global__ void __launch_bounds__(Cfg<DK, DV, kFmt, T, kPro, kOne>::NT, Cfg<DK, DV, kFmt, T, kPro, kOne>::CTAS)
    decode_q8_kernel(const __grid_constant__ Params p, const __grid_constant__ Q8Args a, const __grid_constant__ Ring ring) {
    using C = Cfg<DK, DV, kFmt, T, kPro, kOne>;
    constexpr int W = C::W, RW = C::RW, CPL = C::CPL, G = C::G, PR = DK / 8;  // PR: rows of a partial sum
    using Wd = typename Word<CPL>::type;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ __align__(16) float red[2][2][W][DV];     // [token parity][r | p][warp][column]
    __shared__ __align__(16) float dsum[2][W][4];        // q . e, q . k, |q|^2, |k|^2 of a warp's rows
    __shared__ __align__(16) float rows[W][6][RW];       // k g, q g, g, k, -e; row maxima, then 1 / scale
    __shared__ __align__(16) int4 head[C::MAX_STAGES];   // 0 (-1: no more items), n, h, slot written
    __shared__ __align__(16) int4 next;                  // the next item to bring: item, slot, slot written
    __shared__ __align__(8) int2 piece[8];               // bytes and place in the stage of the 8 copies
    __shared__ __align__(8) uint64_t full[C::MAX_STAGES];
    __shared__ int issued;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n_tok = kOne ? 1 : p.n_tok, n_items = p.n_seq * p.h_v;
    const uint32_t full0 = tc::smem_u32(full), dsm0 = tc::smem_u32(dsm);

    // Producer (warp 0). The next active item and its slots are looked up one issue ahead, and kept
    // in shared memory: registers are what this kernel is short of.
    auto look = [&](int it) {
        int slot = -1, out = -1;
        for (; it < n_items; it += gridDim.x) {
            const int n = it / p.h_v;
            slot = p.slots ? p.slots[n] : n;
            if (slot >= 0 && slot < p.n_slots) {
                out = a.slots_out ? a.slots_out[n] : slot;
                break;
            }
        }
        next = make_int4(it, slot, out, 0);
    };
    auto issue = [&](int i) {  // the i-th of this CTA
        const int4 nx = next;
        if (nx.x < 0) return;
        const int s = i % ring.stages;
        const uint32_t bar = full0 + 8 * s;
        const bool none = nx.x >= n_items;
        const int n = nx.x / p.h_v, h = nx.x % p.h_v;
        if (lane == 0) {
            issued = i + 1;
            head[s] = make_int4(none ? -1 : 0, n, h, nx.z);
            if (none) tc::mbar_arrive(bar);
            else tc::mbar_expect_tx(bar, C::TOK + n_tok * C::REC);
        }
        __syncwarp();
        if (!none && lane < 8) {  // lane c brings piece c
            const int2 pc = piece[lane];
            const size_t row = (size_t)n * n_tok;
            const size_t idx = lane < 2 ? (size_t)nx.y * p.h_v + h : lane < 4 ? row * p.h_qk + h / (p.h_v / p.h_qk) : row * p.h_v + h;
            const char* src = static_cast<const char*>(ring.src[lane]) + idx * pc.x;
            uint32_t dst = dsm0 + s * ring.stage_bytes + pc.y;
            const size_t step = (size_t)(lane < 4 ? p.h_qk : p.h_v) * pc.x;
            bulk_load(dst, src, pc.x, bar);
            if (!kOne && lane >= 2)
                for (int t = 1; t < n_tok; ++t) bulk_load(dst += C::REC, src += step, pc.x, bar);
        }
        if (lane == 0) {
            if (none) next.x = -1;
            else look(nx.x + gridDim.x);
        }
        __syncwarp();
    };

    if (tid == 0) {
        for (int s = 0; s < ring.stages; ++s) tc::mbar_init(full0 + 8 * s, 1);
        tc::fence_mbar_init();
        issued = 0;
        const int bytes[8] = {DK * DV, DK * 4, DK * C::ES, DK * C::ES, DK * C::ES, C::AB, DV * C::ES, DV * C::ES};
        const int place[8] = {0, DK * DV, C::TOK + C::RK, C::TOK + C::RQ, C::TOK + C::RB, C::TOK + C::RA, C::TOK + C::RV, C::TOK + C::RWR};
#pragma unroll
        for (int c = 0; c < 8; ++c) piece[c] = make_int2(bytes[c], place[c]);
        look(blockIdx.x);
    }
    __syncthreads();
    if (warp == 0 && !p.test_withhold_loads)
        for (int s = 0; s + 1 < ring.stages; ++s) issue(s);

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
        const uint8_t* mine = stage + warp * (RW * DV) + c0;  // this lane's columns of the warp's rows
        const uint8_t* rec = stage + C::TOK;
        // values of the codes of rows 2i and 2i + 1, as pairs
        auto values = [&](int i, f32x2* x) {
            q8_unpack_pair<kFmt, CPL>(*reinterpret_cast<const Wd*>(mine + 2 * i * DV), *reinterpret_cast<const Wd*>(mine + (2 * i + 1) * DV), x);
        };
        f32x2 v[G / 2][CPL];
        if (!kOne) {
#pragma unroll
            for (int i = 0; i < RW / 2; ++i) values(i, v[i]);
        }
        for (int t = 0; t < n_tok; ++t, rec += C::REC, buf ^= 1) {
            // the warp's row factors
            __syncwarp();
            float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
            if (RW == 32 || lane < RW) {
                const int i = warp * RW + lane;
                const float kv = to_f32(reinterpret_cast<const T*>(rec + C::RK)[i]), qv = to_f32(reinterpret_cast<const T*>(rec + C::RQ)[i]);
                float bv = to_f32(reinterpret_cast<const T*>(rec + C::RB)[i]);
                float g;
                if (kPro) {
                    g = sigmoid_f(-to_f32(reinterpret_cast<const T*>(rec + C::RA)[i]));
                    bv = sigmoid_f(bv);
                } else {
                    g = expf(reinterpret_cast<const float*>(rec + C::RA)[i]);
                }
                if (t == 0) g *= reinterpret_cast<const float*>(stage + DK * DV)[i];
                const float e = bv * kv;
                rv[0][lane] = kv * g;
                rv[1][lane] = qv * g;
                rv[2][lane] = g;
                rv[3][lane] = kv;
                rv[4][lane] = -e;
                // __fmul_rn: not contracted with the sums below, so that all forms round alike
                d0 = __fmul_rn(qv, e);
                d1 = __fmul_rn(qv, kv);
                if (kPro) {
                    d2 = __fmul_rn(qv, qv);
                    d3 = __fmul_rn(kv, kv);
                }
            }
#pragma unroll
            for (int s_ = 0; (1 << s_) < RW; ++s_) {  // within a partial sum's rows, then over its two
                const int off = (1 << s_) < PR ? (PR / 2) >> s_ : PR;
                d0 += __shfl_xor_sync(0xffffffffu, d0, off);
                d1 += __shfl_xor_sync(0xffffffffu, d1, off);
                if (kPro) {
                    d2 += __shfl_xor_sync(0xffffffffu, d2, off);
                    d3 += __shfl_xor_sync(0xffffffffu, d3, off);
                }
            }
            if (lane == 0) *reinterpret_cast<float4*>(dsum[buf][warp]) = make_float4(d0, d1, d2, d3);
            __syncwarp();

            f32x2 r2[CPL], p2[CPL];
            Cols<float, CPL> rs, ps;
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {
#pragma unroll
                for (int j = 0; j < CPL; ++j)
                    if (i % (PR / 4) == 0) r2[j] = p2[j] = 0ull;
                const ulonglong2 kg = pairs(&rv[0][4 * i]), qg = pairs(&rv[1][4 * i]);
                f32x2 y[2][CPL];
                if (i < RW / 4 - G / 4) {
                    values(2 * i, y[0]);
                    values(2 * i + 1, y[1]);
                } else if (kOne) {  // the last G rows stay in registers
                    values(2 * i, v[(2 * i) % (G / 2)]);
                    values(2 * i + 1, v[(2 * i + 1) % (G / 2)]);
                }
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    const bool kept = i >= RW / 4 - G / 4;
                    const f32x2 y0 = kept ? v[(2 * i) % (G / 2)][j] : y[0][j], y1 = kept ? v[(2 * i + 1) % (G / 2)][j] : y[1][j];
                    r2[j] = fma2(kg.x, y0, r2[j]);
                    p2[j] = fma2(qg.x, y0, p2[j]);
                    r2[j] = fma2(kg.y, y1, r2[j]);
                    p2[j] = fma2(qg.y, y1, p2[j]);
                    if (i % (PR / 4) == PR / 4 - 1) {
                        const float2 ra = unpack2(r2[j]), pa = unpack2(p2[j]);
                        rs.x[j] = i < PR / 4 ? ra.x + ra.y : rs.x[j] + (ra.x + ra.y);
                        ps.x[j] = i < PR / 4 ? pa.x + pa.y : ps.x[j] + (pa.x + pa.y);
                    }
                }
            }
            *reinterpret_cast<Cols<float, CPL>*>(&red[buf][0][warp][c0]) = rs;
            *reinterpret_cast<Cols<float, CPL>*>(&red[buf][1][warp][c0]) = ps;
            // every warp's sums are in; every warp is done with the previous item, too
            if (__syncthreads_or(fault)) {
                fault = true;
                break;
            }
            if (t == 0 && warp == 0) issue(taken + ring.stages - 1);
            f32x2 rc[CPL / 2];
            sum_warps<CPL>(red[buf][0], c0, rc);
            // fused pre-processing: q and k enter unnormalised, and each sum takes its norms here
            float nq = 1.f, nk = 1.f;
            if (kPro) {
                nq = 1.f / fmaxf(sqrtf(sum_dots(dsum[buf], 2)), kL2NormEps);
                nk = 1.f / fmaxf(sqrtf(sum_dots(dsum[buf], 3)), kL2NormEps);
            }
            const size_t row = ((size_t)hd.y * n_tok + t) * p.h_v + hd.z;
            const Cols<T, CPL> wc = reinterpret_cast<const Cols<T, CPL>*>(rec + C::RWR)[lane], vc = reinterpret_cast<const Cols<T, CPL>*>(rec + C::RV)[lane];
            float x[CPL], r[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const float2 rr = unpack2(rc[j / 2]);
                const float wv = to_f32(wc.x[j]);
                x[j] = nk * ((kPro ? sigmoid_f(wv) : wv) * to_f32(vc.x[j]));
                r[j] = nk * (j % 2 ? rr.y : rr.x);
            }
            if (warp == ((taken + t) & (W - 1))) {  // one warp, another each time, writes the outputs
                f32x2 pc[CPL / 2];
                sum_warps<CPL>(red[buf][1], c0, pc);
                const float qe = sum_dots(dsum[buf], 0), qk = sum_dots(dsum[buf], 1);
                float o[CPL];
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    const float2 pp = unpack2(pc[j / 2]);
                    o[j] = __fmul_rn(nq, fmaf(qk, x[j], fmaf(-__fmul_rn(nk, qe), r[j], j % 2 ? pp.y : pp.x)));
                }
                if (a.o_bf16) {
                    Cols<__nv_bfloat16, CPL> ob;
#pragma unroll
                    for (int j = 0; j < CPL; ++j) ob.x[j] = __float2bfloat16_rn(o[j]);
                    *reinterpret_cast<Cols<__nv_bfloat16, CPL>*>(static_cast<__nv_bfloat16*>(p.o) + row * DV + c0) = ob;
                } else {
                    Cols<float, CPL> of;
#pragma unroll
                    for (int j = 0; j < CPL; ++j) of.x[j] = o[j];
                    *reinterpret_cast<Cols<float, CPL>*>(static_cast<float*>(p.o) + row * DV + c0) = of;
                }
            }
            const bool last = t + 1 == n_tok, keep = last && hd.w >= 0 && hd.w < p.n_slots;
            f32x2 xx[CPL], rr[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                xx[j] = pack2(x[j], x[j]);
                rr[j] = pack2(nk * r[j], nk * r[j]);
            }
            // the new state, G rows at a time
            constexpr int kPasses = RW / G;
#pragma unroll  // the second pass's reads beside the first one's scales: 81.2 -> 79.9 us
            for (int ps_ = 0; ps_ < kPasses; ++ps_) {
                const int i0 = (kPasses - 1 - ps_) * G;
#pragma unroll
                for (int i = 0; i < G / 4; ++i) {
                    const ulonglong2 g4 = pairs(&rv[2][i0 + 4 * i]), k4 = pairs(&rv[3][i0 + 4 * i]), e4 = pairs(&rv[4][i0 + 4 * i]);
                    if (kPasses > 1 && ps_ > 0) {
                        values(i0 / 2 + 2 * i, v[2 * i]);
                        values(i0 / 2 + 2 * i + 1, v[2 * i + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        v[2 * i][j] = fma2(g4.x, v[2 * i][j], fma2(k4.x, xx[j], mul2(e4.x, rr[j])));
                        v[2 * i + 1][j] = fma2(g4.y, v[2 * i + 1][j], fma2(k4.y, xx[j], mul2(e4.y, rr[j])));
                    }
                }
                if (kOne ? !keep : !(keep || a.code_steps)) continue;

                // quantise: the row maxima, then one row's scale per lane
                float m[G];
#pragma unroll
                for (int i = 0; i < G / 2; ++i) {
                    float2 y[CPL];
#pragma unroll
                    for (int j = 0; j < CPL; ++j) y[j] = unpack2(v[i][j]);
                    if (CPL == 4) {
                        m[2 * i] = amax_nan(amax_nan(y[0].x, y[1].x, y[2 % CPL].x), y[3 % CPL].x);
                        m[2 * i + 1] = amax_nan(amax_nan(y[0].y, y[1].y, y[2 % CPL].y), y[3 % CPL].y);
                    } else {
                        m[2 * i] = amax_nan(y[0].x, y[1].x);
                        m[2 * i + 1] = amax_nan(y[0].y, y[1].y);
                    }
                }
#pragma unroll
                for (int i = 0; i < G; ++i) m[i] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[i])));
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < G / 4; ++i)
                        *reinterpret_cast<float4*>(&rv[5][i0 + 4 * i]) = make_float4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
                }
                __syncwarp();
                float scale, inv;
                q8_scale<kFmt>(rv[5][i0 + lane % G], scale, inv);
                // (every lane takes a scale, some the same: a branch around it cost 1 %)
                if (kOne) {
                    __syncwarp();
                    rv[5][i0 + lane % G] = inv;
                    __syncwarp();
                }
                const auto inv_of = [&](int i) {  // of rows i and i + 1; kOne 80.0 us this way, 83 by shuffles, the other form 84.7 and 83.2
                    return kOne ? *reinterpret_cast<const f32x2*>(&rv[5][i0 + i]) : pack2(__shfl_sync(0xffffffffu, inv, i), __shfl_sync(0xffffffffu, inv, i + 1));
                };
                const bool zero_rows = __any_sync(0xffffffffu, inv == 0.f);
                uint32_t word[G];
#pragma unroll
                for (int i = 0; i < G / 4; ++i) {
                    q8_pack_pair<kFmt, CPL>(v[2 * i], inv_of(4 * i), word[4 * i], word[4 * i + 1]);
                    q8_pack_pair<kFmt, CPL>(v[2 * i + 1], inv_of(4 * i + 2), word[4 * i + 2], word[4 * i + 3]);
                }
                if (zero_rows) {  // rows whose codes are 0 whatever they hold
#pragma unroll
                    for (int i = 0; i < G; ++i) word[i] = (kOne ? rv[5][i0 + i] : __shfl_sync(0xffffffffu, inv, i)) == 0.f ? 0u : word[i];
                }
                auto put = [&](void* codes, float* sc, size_t state) {
                    const size_t r0 = state * DK + warp * RW + i0;
                    uint8_t* at = static_cast<uint8_t*>(codes) + r0 * DV + c0;
#pragma unroll
                    for (int i = 0; i < G; ++i) *reinterpret_cast<Wd*>(at + i * DV) = (Wd)word[i];
                    if (lane < G) sc[r0 + lane] = scale;
                };
                if (!kOne && a.code_steps) put(a.code_steps, a.scale_steps, row);
                if (keep) put(a.codes, a.scales, (size_t)hd.w * p.h_v + hd.z);
            }
        }
        if (fault) break;
    }
    if (fault && tid == 0) {
        atomicOr(&g_status_q8, kStatusWaitTimeout);
        // give loads still in flight a last bounded chance to land before the CTA exits
        for (int i = taken; i < issued; ++i) tc::mbar_wait(full0 + 8 * (i % ring.stages), (i / ring.stages) & 1, p.wait_ns);
    }
}

template <int DK, int DV, int kFmt, typename T, bool kPro, bool kOne>
cudaError_t launch(const Params& p, const Q8Args& a, cudaStream_t st) {
    using C = Cfg<DK, DV, kFmt, T, kPro, kOne>;
    auto kern = decode_q8_kernel<DK, DV, kFmt, T, kPro, kOne>;
    const auto stage_bytes = [](int n_tok) { return (C::TOK + n_tok * C::REC + 127) & ~127; };
    // three stages (two items ahead) where the SM's CTAs have room for them, else two
    const auto stages = [&](int n_tok) { return C::CTAS * (3 * stage_bytes(n_tok) + 22 * 1024) <= 224 * 1024 ? 3 : 2; };
    const Ring ring{stages(p.n_tok), stage_bytes(p.n_tok),
                    {a.codes, a.scales, p.k, p.q, p.b, kPro ? p.a_raw : static_cast<const void*>(p.log_alpha), p.v, p.w}};
    const int smem = ring.stages * ring.stage_bytes;
    // CTAs that the device holds, looked up once per device and token count: for a small batch these
    // queries take as long as the launch
    constexpr int kDevices = 16;
    static std::atomic<int> resident[kDevices][GDN2_DECODE_MAX_TOKENS + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int ctas = dev < kDevices ? resident[dev][p.n_tok].load(std::memory_order_relaxed) : 0;
    if (ctas == 0) {
        int sms = 0, per_sm = 0, most = 0;
        for (int t = 1; t <= (kOne ? 1 : GDN2_DECODE_MAX_TOKENS); ++t) most = std::max(most, stages(t) * stage_bytes(t));
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::NT, smem);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        ctas = sms * per_sm;
        if (dev < kDevices) resident[dev][p.n_tok].store(ctas, std::memory_order_relaxed);
    }
    const int items = p.n_seq * p.h_v;
    kern<<<std::min(items, ctas), C::NT, smem, st>>>(p, a, ring);
    return cudaGetLastError();
}

template <int DK, int DV, int kFmt, typename T, bool kPro>
cudaError_t launch_n(const Params& p, const Q8Args& a, cudaStream_t st) {
    return p.n_tok == 1 && !a.code_steps ? launch<DK, DV, kFmt, T, kPro, true>(p, a, st) : launch<DK, DV, kFmt, T, kPro, false>(p, a, st);
}

template <int DK, int DV, int kFmt>
cudaError_t launch_t(const Params& p, const Q8Args& a, cudaStream_t st) {
    if (a.bf16) return p.prologue ? launch_n<DK, DV, kFmt, __nv_bfloat16, true>(p, a, st) : launch_n<DK, DV, kFmt, __nv_bfloat16, false>(p, a, st);
    return p.prologue ? launch_n<DK, DV, kFmt, float, true>(p, a, st) : launch_n<DK, DV, kFmt, float, false>(p, a, st);
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
