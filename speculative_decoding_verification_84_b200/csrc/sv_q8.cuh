// sv_q8.cuh -- the draft's head in 8-bit integers: root-mean-square norm with the
// residual's addition to int8 rows with a scale each (sv_q8_rows), and the int8
// product with a scale for each token and channel (sv_q8_gemm).
//
// Rows to int8.  s = x + r, p = s w, a = max |p|: q = round(127 p / a) (ties to
// even), scale = a / (127 rms), rms = sqrt(mean(s^2) + eps).  The norm's factor
// cancels out of q, so one reduction gives everything: sum s^2 and max |p|.  Sums
// are fp32 (fp64 where they leave its range), q is the integer that the formula
// gives in fp64: fp32 decides all values but those within 1e-4 of a half (its
// error is below 6 * 2^-24 * 127 = 5e-5), and those are decided in fp64, against
// the fp64 maximum.  A second pair of roundings would make such a value depend on
// the order of the row's sum.
//   sv_q8_rows       a row in registers, blockDim.x threads a row
//   sv_q8_rows_long  rows beyond that: read three times, fp64 throughout
//
// The product.  z[m][v] = sa[m] sw[v] sum_k a[m][k] w[v][k] on the tensor cores
// (tcgen05 kind::i8, s32 accumulators: exact for K <= 131056, 127 * 128 * K and
// 128 * 128 * K both below 2^31).  The weights are the MMA's 128 rows and the
// tokens its columns, so a small batch pads to 16 tokens, not to 128, and every
// weight byte crosses to an SM once per token tile (up to 256 tokens).
//   warp 0 (one thread)  TMA: 128 x 128 bytes of weights and nt x 128 of tokens per
//                        stage, 128-byte swizzle, an mbarrier ring
//   warp 1 (one thread)  tcgen05.mma, M = 128, N = nt, four K = 32 steps per stage
//   warp 2               TMEM columns (two accumulators of nt columns)
//   warps 4-11           epilogue: lane = channel, column = token; scales, rounding,
//                        stores
#pragma once

#include "sv_common.cuh"
#include "sv_tc.cuh"

namespace sv {

// ----------------------------------------------------------------------------- rows to int8

struct Q8RowsArgs {
    const void* x;       // [M][d]
    const void* r;       // [M][d] or null
    const void* w;       // [d] or null (ones)
    int8_t* q;           // [M][ldq]
    float* scale;        // [M]
    void* sum;           // [M][d] or null; may be x or r
    void* normed;        // [M][d] or null
    long long ldq;
    int M, d;
    float eps;
    int norm;            // 0: scale = a / 127 (no norm)
};

template <int ESZ>
__device__ __forceinline__ float q8_ld1(const void* p, size_t i)
{
    if (ESZ == 4) return static_cast<const float*>(p)[i];
    return __uint_as_float((uint32_t) static_cast<const unsigned short*>(p)[i] << 16);
}

template <int ESZ>
__device__ __forceinline__ void q8_st1(void* p, size_t i, float v)
{
    if (ESZ == 4) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ double q8_warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// max of non-negative doubles over the warp (their bits order as integers)
__device__ __forceinline__ double q8_warp_max(double v)
{
    const unsigned hi = (unsigned)__double2hiint(v), lo = (unsigned)__double2loint(v);
    const unsigned h = __reduce_max_sync(0xffffffffu, hi);
    const unsigned l = __reduce_max_sync(0xffffffffu, hi == h ? lo : 0u);
    return __hiloint2double((int)h, (int)l);
}

// Very long rows: one CTA a row, three passes over it.
template <int ESZ>
__global__ void __launch_bounds__(1024) sv_q8_rows_long(Q8RowsArgs g)
{
    __shared__ double s_sum[32], s_max[32];
    __shared__ unsigned s_bad[32];
    const size_t base = (size_t)blockIdx.x * g.d;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    double ss = 0.0, pm = 0.0;
    unsigned top = 0;
    for (int i = threadIdx.x; i < g.d; i += blockDim.x) {
        const float x = q8_ld1<ESZ>(g.x, base + i), r = g.r ? q8_ld1<ESZ>(g.r, base + i) : 0.f;
        const float w = g.w ? q8_ld1<ESZ>(g.w, i) : 1.f;
        top = max(top, __float_as_uint((x + r) * w) & 0x7fffffffu);
        const double s = (double)x + (double)r;
        ss += s * s;
        pm = fmax(pm, fabs(s * (double)w));
    }
    ss = q8_warp_sum(ss);
    pm = q8_warp_max(pm);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) { s_sum[warp] = ss; s_max[warp] = pm; s_bad[warp] = top; }
    __syncthreads();
    ss = q8_warp_sum(lane < nw ? s_sum[lane] : 0.0);
    pm = q8_warp_max(lane < nw ? s_max[lane] : 0.0);
    top = __reduce_max_sync(0xffffffffu, lane < nw ? s_bad[lane] : 0u);
    const bool bad = top >= 0x7f800000u;
    const double rms = g.norm ? sqrt(ss / g.d + (double)g.eps) : 1.0;
    if (threadIdx.x == 0) g.scale[blockIdx.x] = bad ? NAN : (pm > 0.0 ? (float)(pm / (127.0 * rms)) : 0.f);
    for (int i = threadIdx.x; i < g.d; i += blockDim.x) {
        const float x = q8_ld1<ESZ>(g.x, base + i), r = g.r ? q8_ld1<ESZ>(g.r, base + i) : 0.f;
        const float w = g.w ? q8_ld1<ESZ>(g.w, i) : 1.f;
        const double p = ((double)x + (double)r) * (double)w;
        g.q[(size_t)blockIdx.x * g.ldq + i] = (bad || !(pm > 0.0)) ? 0 : (int8_t)(int)rint(p * 127.0 / pm);
        if (g.sum) q8_st1<ESZ>(g.sum, base + i, x + r);
        if (g.normed) q8_st1<ESZ>(g.normed, base + i, bad ? NAN : (pm > 0.0 ? (float)(p / rms) : 0.f));
    }
}

// NV pieces of VEC elements a thread (VEC x ESZ = 16 bytes, or VEC = 1 for rows
// that start at no vector boundary); blockDim.x threads a row, and blockDim.y rows
// a CTA when blockDim.x is one warp (no barrier then).
template <int ESZ, int VEC, int NV>
__global__ void __launch_bounds__(1024) sv_q8_rows(Q8RowsArgs g)
{
    static_assert(VEC == 1 || VEC * ESZ == 16, "a piece is an element or a 16-byte vector");
    __shared__ float s_ss[32];
    __shared__ unsigned s_pm[32];
    __shared__ double s_dm[32];
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= g.M) return;  // only where a row is one warp
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nw = nthr >> 5;
    const size_t base = (size_t)row * g.d;

    // every load first (sum may be written over x or r)
    uint4 xv[VEC > 1 ? NV : 1], rv[VEC > 1 ? NV : 1], wv[VEC > 1 ? NV : 1];
    float x1[VEC > 1 ? 1 : NV], r1[VEC > 1 ? 1 : NV], w1[VEC > 1 ? 1 : NV];
    const uint32_t one = ESZ == 2 ? 0x3f803f80u : 0x3f800000u;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = (j * nthr + tid) * VEC;
        const bool in = i < g.d;
        if (VEC > 1) {
            xv[j] = in ? *reinterpret_cast<const uint4*>(static_cast<const char*>(g.x) + (base + i) * ESZ) : make_uint4(0, 0, 0, 0);
            rv[j] = (in && g.r) ? *reinterpret_cast<const uint4*>(static_cast<const char*>(g.r) + (base + i) * ESZ)
                                : make_uint4(0, 0, 0, 0);
            wv[j] = (in && g.w) ? __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(g.w) + (size_t)i * ESZ))
                                : make_uint4(one, one, one, one);
        } else {
            x1[j] = in ? q8_ld1<ESZ>(g.x, base + i) : 0.f;
            r1[j] = (in && g.r) ? q8_ld1<ESZ>(g.r, base + i) : 0.f;
            w1[j] = (in && g.w) ? q8_ld1<ESZ>(g.w, i) : 1.f;
        }
    }
    auto get = [&](int j, float* x, float* r, float* w) {
        if (VEC > 1) {
            unpack<ESZ>(xv[j], x);
            unpack<ESZ>(rv[j], r);
            unpack<ESZ>(wv[j], w);
        } else {
            x[0] = x1[j];
            r[0] = r1[j];
            w[0] = w1[j];
        }
    };
    float ss = 0.f;
    unsigned tpm = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float x[VEC], r[VEC], w[VEC];
        get(j, x, r, w);
        const int i = (j * nthr + tid) * VEC;
        float s[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[e] = x[e] + r[e];
            ss = fmaf(s[e], s[e], ss);
            tpm = max(tpm, __float_as_uint(s[e] * w[e]) & 0x7fffffffu);
        }
        if (g.sum && i < g.d) {
            if (VEC > 1 && ESZ == 2) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(s[(2 * e) % VEC], s[(2 * e + 1) % VEC]);
                    o[e] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(static_cast<char*>(g.sum) + (base + i) * ESZ) = make_uint4(o[0], o[1], o[2], o[3]);
            } else if (VEC > 1) {
                *reinterpret_cast<float4*>(static_cast<char*>(g.sum) + (base + i) * ESZ) =
                    make_float4(s[0], s[1 % VEC], s[2 % VEC], s[3 % VEC]);
            } else {
                q8_st1<ESZ>(g.sum, base + i, s[0]);
            }
        }
    }
    // sum s^2 and max |p| (as bits: NaN and inf order above every number)
    unsigned pm = __reduce_max_sync(0xffffffffu, tpm);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (nw > 1) {
        if (lane == 0) { s_ss[warp] = ss; s_pm[warp] = pm; }
        __syncthreads();
        ss = lane < nw ? s_ss[lane] : 0.f;
        pm = __reduce_max_sync(0xffffffffu, lane < nw ? s_pm[lane] : 0u);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const bool bad = pm >= 0x7f800000u;
    const float pmf = __uint_as_float(pm);
    const bool tiny = pmf < 0x1p-100f;  // 127 / pmf, or the products themselves, leave fp32: all in fp64
    // the maximum in fp64, over the values that reach the fp32 one to 2^-20
    const float thr = tiny ? 0.f : pmf * (1.f - 0x1p-20f);
    double dm = 0.0;
    if (__uint_as_float(tpm) >= thr && !bad) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[VEC], r[VEC], w[VEC];
            get(j, x, r, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (fabsf((x[e] + r[e]) * w[e]) >= thr) dm = fmax(dm, fabs(((double)x[e] + (double)r[e]) * (double)w[e]));
        }
    }
    dm = q8_warp_max(dm);
    if (nw > 1) {
        if (lane == 0) s_dm[warp] = dm;
        __syncthreads();
        dm = q8_warp_max(lane < nw ? s_dm[lane] : 0.0);
    }
    // the norm; a sum of squares outside fp32's comfortable range is taken again in fp64
    double ms = 1.0;
    if (g.norm) {
        ms = (double)ss / g.d + (double)g.eps;
        if (!bad && (!(ss <= 0x1p120f) || ms < 0x1p-80)) {
            double sd = 0.0;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float x[VEC], r[VEC], w[VEC];
                get(j, x, r, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const double s = (double)x[e] + (double)r[e];
                    sd += s * s;
                }
            }
            sd = q8_warp_sum(sd);
            if (nw > 1) {
                __syncthreads();  // s_dm is read
                if (lane == 0) s_dm[warp] = sd;
                __syncthreads();
                sd = q8_warp_sum(lane < nw ? s_dm[lane] : 0.0);
            }
            ms = sd / g.d + (double)g.eps;
        }
    }
    const bool zero = !(dm > 0.0);
    if (tid == 0) g.scale[row] = bad ? NAN : (zero ? 0.f : (float)(dm / (127.0 * sqrt(ms))));
    const float k = 127.f / pmf;
    const bool wide = tiny || ms < 0x1p-200 || ms > 0x1p200;  // 1 / rms, or p, leaves fp32
    float inv = 0.f;
    if (g.normed) inv = bad ? NAN : (zero ? 0.f : (float)(1.0 / sqrt(ms)));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = (j * nthr + tid) * VEC;
        if (i >= g.d) continue;
        float x[VEC], r[VEC], w[VEC], y[VEC];
        get(j, x, r, w);
        int q[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float p = (x[e] + r[e]) * w[e];
            const float t = p * k, n = rintf(t);
            q[e] = (int)n;
            if (fabsf(t - n) > 0.4999f || tiny) {
                const double pd = ((double)x[e] + (double)r[e]) * (double)w[e];
                q[e] = zero ? 0 : (int)rint(pd * 127.0 / dm);
            }
            if (bad) q[e] = 0;
            y[e] = p * inv;
            if (g.normed && wide && !bad && !zero) y[e] = (float)(((double)x[e] + (double)r[e]) * (double)w[e] / sqrt(ms));
        }
        int8_t* qo = g.q + (size_t)row * g.ldq + i;
        if (VEC == 1) {
            qo[0] = (int8_t)q[0];
        } else {
            uint32_t o[VEC > 4 ? 2 : 1];
#pragma unroll
            for (int h = 0; h < (VEC > 4 ? 2 : 1); ++h)
                o[h] = (uint32_t)(q[(4 * h) % VEC] & 255) | (uint32_t)(q[(4 * h + 1) % VEC] & 255) << 8 |
                       (uint32_t)(q[(4 * h + 2) % VEC] & 255) << 16 | (uint32_t)(q[(4 * h + 3) % VEC] & 255) << 24;
            if (VEC > 4) *reinterpret_cast<uint2*>(qo) = make_uint2(o[0], o[VEC > 4 ? 1 : 0]);
            else *reinterpret_cast<uint32_t*>(qo) = o[0];
        }
        if (g.normed) {
            if (VEC > 1 && ESZ == 2) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(y[(2 * e) % VEC], y[(2 * e + 1) % VEC]);
                    o[e] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(static_cast<char*>(g.normed) + (base + i) * ESZ) = make_uint4(o[0], o[1], o[2], o[3]);
            } else if (VEC > 1) {
                *reinterpret_cast<float4*>(static_cast<char*>(g.normed) + (base + i) * ESZ) =
                    make_float4(y[0], y[1 % VEC], y[2 % VEC], y[3 % VEC]);
            } else {
                q8_st1<ESZ>(g.normed, base + i, y[0]);
            }
        }
    }
}

// ----------------------------------------------------------------------------- the product

constexpr int kQ8BM = 128;        // channels per tile = the MMA's M
constexpr int kQ8BK = 128;        // K per stage: one 128-byte swizzled row of int8
constexpr int kQ8MaxNT = 256;     // tokens per tile = the MMA's N
constexpr int kQ8MaxStages = 12;
constexpr int kQ8EpiWarps = 8;    // per TMEM lane quarter two, on alternate 16-column chunks
constexpr int kQ8Threads = 128 + 32 * kQ8EpiWarps;
constexpr int kQ8SmemMax = 227 * 1024 - 1024;  // dynamic shared memory of one CTA (static part kept apart)
constexpr int kQ8WBytes = kQ8BM * kQ8BK;

struct Q8GemmArgs {
    void* out;             // [M][V], bf16 or f32
    const float* a_scale;  // [M]
    const float* w_scale;  // [V]
    int* err;              // optional: 1 if a wait gave up
    int M, V, K;
    int nt;                // tokens per tile, a multiple of 16
    int m_tiles, v_tiles;
    int stages;
    int tmem_cols;         // a power of two, two accumulators
};

// Instruction descriptor: s32 accumulator, signed 8-bit A and B, both K-major.
__device__ __forceinline__ uint32_t q8_idesc(int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kQ8BM >> 4) << 24);
}

__device__ __forceinline__ void q8_mma(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(tmem_d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u), "r"(0u), "r"(0u));
}

__device__ __forceinline__ void q8_tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Persistent, one CTA per SM; tiles blockIdx.x, blockIdx.x + gridDim.x, ... with
// the token tile fastest, so the CTAs that share weights run at about the same time.
// Every wait on an mbarrier is bounded: past kLrPolls polls the CTA raises *err,
// stops issuing, and still frees its TMEM.
template <int ESZ>
__global__ void __launch_bounds__(kQ8Threads, 1)
    sv_q8_gemm(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ta, Q8GemmArgs g)
{
    extern __shared__ unsigned char q8_dyn[];
    // every stage starts on a 1024-byte boundary of the shared window (the swizzle atom)
    unsigned char* ring = q8_dyn + ((1024u - (lr_smem(q8_dyn) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full[kQ8MaxStages], empty[kQ8MaxStages], tfull[2], tempty[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_consumed;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kbs = (g.K + kQ8BK - 1) / kQ8BK, S = g.stages;
    const int STAGE = kQ8WBytes + g.nt * kQ8BK;
    const long long tiles = (long long)g.m_tiles * g.v_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            lr_mbar_init(&full[s], 1);
            lr_mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            lr_mbar_init(&tfull[b], 1);
            lr_mbar_init(&tempty[b], kQ8EpiWarps);
        }
        s_abort = 0;
        s_consumed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(lr_smem(&s_tmem)),
                     "r"(g.tmem_cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    lr_fence_before();
    __syncthreads();
    lr_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* abort = &s_abort;

    int issued = 0;
    if (warp == 0 && lane == 0) {
        // ---- producer: one global count of stages across the CTA's tiles
        int it = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const int m0 = (int)(t % g.m_tiles) * g.nt, v0 = (int)(t / g.m_tiles) * kQ8BM;
            for (int kb = 0; kb < kbs; ++kb, ++it) {
                const int s = it % S;
                if (it >= S && !lr_wait(&empty[s], (unsigned)(it / S - 1) & 1u, abort, g.err)) { ok = false; break; }
                unsigned char* st = ring + s * STAGE;
                lr_expect_tx(&full[s], (unsigned)STAGE);
                lr_tma_2d(st, &tw, &full[s], kb * kQ8BK, v0);
                lr_tma_2d(st + kQ8WBytes, &ta, &full[s], kb * kQ8BK, m0);
                issued = it + 1;
            }
        }
    } else if (warp == 1 && lane == 0) {
        // ---- MMA issuer
        const uint32_t idesc = q8_idesc(g.nt);
        int it = 0, i = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++i) {
            const int b = i & 1, use = i >> 1;
            if (use >= 1 && !lr_wait(&tempty[b], (unsigned)(use - 1) & 1u, abort, g.err)) break;
            lr_fence_after();
            const uint32_t d = tmem + (uint32_t)(b * (g.tmem_cols / 2));
            for (int kb = 0; kb < kbs; ++kb, ++it) {
                const int s = it % S;
                if (!lr_wait(&full[s], (unsigned)(it / S) & 1u, abort, g.err)) { ok = false; break; }
                lr_fence_after();
                const uint32_t w0 = lr_smem(ring + s * STAGE), a0 = w0 + kQ8WBytes;
#pragma unroll
                for (int j = 0; j < kQ8BK / 32; ++j)  // K = 32 per MMA: 32 bytes along the swizzled row
                    q8_mma(d, lr_desc(w0 + 32 * j), lr_desc(a0 + 32 * j), idesc, (kb > 0 || j > 0) ? 1u : 0u);
                lr_commit(&empty[s]);
                s_consumed = it + 1;
            }
            lr_commit(&tfull[b]);
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp 4 + e owns TMEM lanes (= channels of the tile) 32q .. 32q + 31,
        // q = e % 4, and the 16-column chunks e / 4, e / 4 + 2, ...
        const int q = (warp - 4) & 3, grp = (warp - 4) >> 2;
        int i = 0;
        for (long long t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            const int b = i & 1, use = i >> 1;
            const int m0 = (int)(t % g.m_tiles) * g.nt;
            const int v = (int)(t / g.m_tiles) * kQ8BM + 32 * q + lane;
            const float sw = v < g.V ? __ldg(g.w_scale + v) : 0.f;
            // one lane waits, so the warp-wide tcgen05.ld below runs on all lanes or none
            int ready = 0;
            if (lane == 0) ready = lr_wait(&tfull[b], (unsigned)use & 1u, abort, g.err) ? 1 : 0;
            ready = __shfl_sync(0xffffffffu, ready, 0);
            if (!ready) break;
            lr_fence_after();
            const uint32_t acc = tmem + (uint32_t)(b * (g.tmem_cols / 2)) + ((uint32_t)(32 * q) << 16);
            for (int c = grp * 16; c < g.nt && m0 + c < g.M; c += 32) {
                uint32_t r[16];
                q8_tmem_ld16(acc + (uint32_t)c, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int m = m0 + c + j;
                    if (m < g.M && v < g.V) {
                        const float z = (float)(int)r[j] * (__ldg(g.a_scale + m) * sw);
                        q8_st1<ESZ>(g.out, (size_t)m * g.V + v, z);
                    }
                }
            }
            lr_fence_before();
            __syncwarp();
            if (lane == 0) lr_arrive(&tempty[b]);
        }
    }
    lr_fence_before();
    __syncthreads();
    // after a wait gave up: let the copies this CTA issued but never consumed land
    // (bounded) before its shared memory goes away
    if (warp == 0 && lane == 0 && s_abort) {
        for (int it = s_consumed; it < issued; ++it) {
            const unsigned par = (unsigned)(it / S) & 1u;
            for (unsigned k = 0; k < kLrPolls && !lr_try_wait(&full[it % S], par); ++k) {
            }
        }
    }
    if (warp == 2) {
        lr_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_cols));
    }
}

}  // namespace sv
