// decode_q8.cu -- decode on an 8-bit state pool (q8.cuh): n_tok new tokens per sequence, each
// state read as codes, advanced in fp32 and quantised as it is written.
//
// One CTA of 256 threads owns one (sequence, value head); the arithmetic is decode.cu's:
//   r = (Diag(alpha) S)^T k,  p = (Diag(alpha) S)^T q
//   S <- Diag(alpha) S - (b (.) k) r^T + k x^T,   o = p - (q . (b (.) k)) r + (q . k) x
// Between the tokens of one call the state stays in fp32 registers; only what is written to the
// pool, or to the per-token states, is rounded.
#include "q8.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float tok_f32(const void* p, size_t i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

template <int DK, int DV, int kFmt>
__global__ void __launch_bounds__(kThreads) decode_q8_kernel(const __grid_constant__ Params p, const __grid_constant__ Q8Args a) {
    constexpr int TPR = DV / 4, RG = kThreads / TPR, RPT = DK / RG;
    __shared__ float sa[DK], sk[DK], sq[DK], se[DK], sx[DV];
    __shared__ float4 red[2][RG][TPR];  // [r | p]
    __shared__ float dots[4];           // q . e, q . k, |q|^2, |k|^2

    const int n = blockIdx.x / p.h_v, h = blockIdx.x % p.h_v, g = h / (p.h_v / p.h_qk);
    const int slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.n_slots) return;  // an inactive sequence: nothing to do
    const int out = a.slots_out ? a.slots_out[n] : slot;
    const int cg = threadIdx.x % TPR, rg = threadIdx.x / TPR, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t* codes = static_cast<const uint32_t*>(a.codes);

    float4 s[RPT];
    {
        const size_t row0 = ((size_t)slot * p.h_v + h) * DK;
        uint32_t c[RPT];
        float sc[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            c[i] = codes[(row0 + rg + RG * i) * TPR + cg];
            sc[i] = a.scales[row0 + rg + RG * i];
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float4 x = q8_unpack<kFmt>(c[i]);
            s[i] = make_float4(x.x * sc[i], x.y * sc[i], x.z * sc[i], x.w * sc[i]);
        }
    }
    auto write = [&](uint32_t* wc, float* ws) {  // rows of one state, quantised
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            uint32_t m = max(max(mag_bits(s[i].x), mag_bits(s[i].y)), max(mag_bits(s[i].z), mag_bits(s[i].w)));
#pragma unroll
            for (int off = TPR / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
            float scale, inv;
            q8_scale<kFmt>(__uint_as_float(m), scale, inv);
            wc[(rg + RG * i) * TPR + cg] = q8_pack<kFmt>(s[i], inv);
            if (cg == 0) ws[rg + RG * i] = scale;
        }
    };

    for (int t = 0; t < p.n_tok; ++t) {
        const size_t row = (size_t)n * p.n_tok + t, tq = row * p.h_qk + g, tv = row * p.h_v + h;
        for (int c = threadIdx.x; c < DK; c += kThreads) {
            const float kv = tok_f32(p.k, tq * DK + c, a.bf16), bv = tok_f32(p.b, tv * DK + c, a.bf16);
            sk[c] = kv;
            sq[c] = tok_f32(p.q, tq * DK + c, a.bf16);
            sa[c] = p.prologue ? sigmoid_f(-tok_f32(p.a_raw, tv * DK + c, a.bf16)) : expf(p.log_alpha[tv * DK + c]);
            se[c] = (p.prologue ? sigmoid_f(bv) : bv) * kv;
        }
        for (int c = threadIdx.x; c < DV; c += kThreads) {
            const float wv = tok_f32(p.w, tv * DV + c, a.bf16);
            sx[c] = (p.prologue ? sigmoid_f(wv) : wv) * tok_f32(p.v, tv * DV + c, a.bf16);
        }
        __syncthreads();
        if (warp == 0) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c = lane; c < DK; c += 32) {
                d[0] += sq[c] * se[c];
                d[1] += sq[c] * sk[c];
                d[2] += sq[c] * sq[c];
                d[3] += sk[c] * sk[c];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += __shfl_xor_sync(0xffffffffu, d[j], off);
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) dots[j] = d[j];
            }
        }
        __syncthreads();
        // fused pre-processing: q and k are divided by their norms where they are used
        const float nq = p.prologue ? 1.f / fmaxf(sqrtf(dots[2]), kL2NormEps) : 1.f;
        const float nk = p.prologue ? 1.f / fmaxf(sqrtf(dots[3]), kL2NormEps) : 1.f;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f), pq = r;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int rw = rg + RG * i;
            const float al = sa[rw], kv = sk[rw] * nk, qv = sq[rw] * nq;
            s[i].x *= al; s[i].y *= al; s[i].z *= al; s[i].w *= al;
            r.x = fmaf(kv, s[i].x, r.x); r.y = fmaf(kv, s[i].y, r.y);
            r.z = fmaf(kv, s[i].z, r.z); r.w = fmaf(kv, s[i].w, r.w);
            pq.x = fmaf(qv, s[i].x, pq.x); pq.y = fmaf(qv, s[i].y, pq.y);
            pq.z = fmaf(qv, s[i].z, pq.z); pq.w = fmaf(qv, s[i].w, pq.w);
        }
        red[0][rg][cg] = r;
        red[1][rg][cg] = pq;
        __syncthreads();
        r = make_float4(0.f, 0.f, 0.f, 0.f);
        pq = r;
#pragma unroll
        for (int j = 0; j < RG; ++j) {
            const float4 x = red[0][j][cg], y = red[1][j][cg];
            r.x += x.x; r.y += x.y; r.z += x.z; r.w += x.w;
            pq.x += y.x; pq.y += y.y; pq.z += y.z; pq.w += y.w;
        }
        const float4 x = *reinterpret_cast<const float4*>(&sx[4 * cg]);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int rw = rg + RG * i;
            const float e = -se[rw] * nk, kv = sk[rw] * nk;
            s[i].x = fmaf(kv, x.x, fmaf(e, r.x, s[i].x));
            s[i].y = fmaf(kv, x.y, fmaf(e, r.y, s[i].y));
            s[i].z = fmaf(kv, x.z, fmaf(e, r.z, s[i].z));
            s[i].w = fmaf(kv, x.w, fmaf(e, r.w, s[i].w));
        }
        if (rg == 0) {
            const float qe = dots[0] * nq * nk, qk = dots[1] * nq * nk;
            const float4 o = make_float4(pq.x - qe * r.x + qk * x.x, pq.y - qe * r.y + qk * x.y, pq.z - qe * r.z + qk * x.z,
                                         pq.w - qe * r.w + qk * x.w);
            const size_t at = tv * DV + 4 * cg;
            if (a.o_bf16) {
                __nv_bfloat162* ob = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.o) + at);
                ob[0] = __floats2bfloat162_rn(o.x, o.y);
                ob[1] = __floats2bfloat162_rn(o.z, o.w);
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) = o;
            }
        }
        if (a.code_steps) write(static_cast<uint32_t*>(a.code_steps) + tv * (DK * TPR), a.scale_steps + tv * DK);
        __syncthreads();  // the token's vectors and sums have been read
    }
    if (out >= 0 && out < p.n_slots) {
        const size_t row0 = ((size_t)out * p.h_v + h) * DK;
        write(static_cast<uint32_t*>(a.codes) + row0 * TPR, a.scales + row0);
    }
}

template <int DK, int DV>
cudaError_t launch(const Params& p, const Q8Args& a, cudaStream_t st) {
    const int grid = p.n_seq * p.h_v;
    if (a.fmt == GDN2_Q8_INT8)
        decode_q8_kernel<DK, DV, GDN2_Q8_INT8><<<grid, kThreads, 0, st>>>(p, a);
    else
        decode_q8_kernel<DK, DV, GDN2_Q8_E4M3><<<grid, kThreads, 0, st>>>(p, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_q8(const Params& p, const Q8Args& a, cudaStream_t st) {
    if (p.dk == 128) return p.dv == 128 ? launch<128, 128>(p, a, st) : launch<128, 64>(p, a, st);
    return p.dv == 128 ? launch<64, 128>(p, a, st) : launch<64, 64>(p, a, st);
}

}  // namespace gdn2
