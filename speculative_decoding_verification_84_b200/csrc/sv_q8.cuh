// sv_q8.cuh -- the draft's head in 8-bit integers: root-mean-square norm with the
// residual's addition to int8 rows with a scale each (sv_q8_rows), and the int8
// product with a scale for each token and channel (sv_q8_gemm).
//
// Rows to int8.  s = x + r, p = s w, a = max |p|: q = round(127 p / a) (ties to
// even), scale = a / (127 rms), rms = sqrt(mean(s^2) + eps).  The norm's factor
// cancels out of q, so one reduction gives everything: sum s^2 and max |p|.  Sums
// are fp32 (fp64 where they leave its range), q is the integer that the formula
// gives in fp64: fp32 decides all values but those that its roundings leave within
// reach of a half, and those are decided in fp64, against the fp64 maximum.
//   sv_q8_rows       CTAs walk rows, the next one on its way to shared memory
//   sv_q8_rows_long  rows that shared memory cannot hold three of: read twice from
//                    memory, fp64 throughout
// Bound by bytes and instructions: 16384 x 4096 bf16 with a residual takes 93 us, 5.0
// TB/s of the 470 MB it cannot do without.
//
// The product.  z[m][v] = sa[m] sw[v] sum_k a[m][k] w[v][k] on the tensor cores
// (tcgen05 kind::i8, s32 accumulators: exact for K <= 131056, 127 * 128 * K and
// 128 * 128 * K both below 2^31).  The weights are the MMA's 128 rows and the
// tokens its columns, so a small batch pads to 16 tokens, not to 128, and every
// weight byte crosses to an SM once per token tile (up to 256 tokens; 320 in a tile of
// two).  Bound by the weights' bytes up to some 250 tokens (1 x 4096 x 128256: 82 us, 6.4
// TB/s), above by the tensor cores at the power limit (2048 x 4096 x 151936: 800 us, 3.2
// P operations a second; at 32000 columns the tensor pipe is active for 81 %).
//   warp 0     TMA: per stage two K blocks of 128 x 128 bytes of weights and nt x 128 of
//              tokens, 128-byte swizzle, an mbarrier ring
//   warp 1     tcgen05.mma, M = 128 (256 on a pair of SMs), N = nt, K = 32 each
//   warp 2     TMEM columns (up to four accumulators of nt columns)
//   warps 4-19 epilogue: lane = channel, column = token; scales, rounding, stores
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

// 16 / ESZ values rounded and packed into 16 bytes.
template <int ESZ>
__device__ __forceinline__ uint4 q8_pack(const float* v)
{
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[(2 * e) % (16 / ESZ)], v[(2 * e + 1) % (16 / ESZ)]);
        o[e] = ESZ == 4 ? __float_as_uint(v[e]) : *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
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

// Very long rows: one CTA a row, two passes over it, one element at a time (4096 x 16384 f32
// with a residual: 472-500 us, 0.9 GB of it: 133 us at the copy's rate).
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

__device__ __forceinline__ int cdiv_pos(int a, int b) { return a > 0 ? (a + b - 1) / b : 0; }

// 16 bytes of shared memory, of which `bytes` are read and the rest are zero.
__device__ __forceinline__ void q8_cp16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// max(m, |a|, |b|); a NaN stays
__device__ __forceinline__ float q8_max3(float m, float a, float b)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}

// A 16-byte vector's elements as packed fp32 pairs.
template <int ESZ, int P>
__device__ __forceinline__ void q8_pairs(const uint4& v, unsigned long long (&p)[P])
{
    float x[16 / ESZ];
    unpack<ESZ>(v, x);
#pragma unroll
    for (int e = 0; e < P; ++e) p[e] = pack2(x[2 * e], x[2 * e + 1]);
}

// A row in shared memory: element e of piece j of the row's thread t, in fp64.
template <int ESZ, bool RES, bool AL>
struct Q8Row {
    static constexpr int VEC = 16 / ESZ;
    const Q8RowsArgs& g;
    const unsigned char* x;  // the row's first element
    int residual;            // bytes from there to the residual's
    __device__ __forceinline__ int index(int j, int t) const { return (j * (int)blockDim.x + t) * VEC; }
    __device__ __forceinline__ double sum(int i) const
    {
        const double v = q8_ld1<ESZ>(x, i);
        return RES ? v + (double)q8_ld1<ESZ>(x + residual, i) : v;
    }
    __device__ __forceinline__ double prod(int i) const { return sum(i) * (g.w ? (double)q8_ld1<ESZ>(g.w, i) : 1.0); }
    // elements i .. i + VEC in fp32, the products as the kernel forms them; 0 past the row
    __device__ __forceinline__ void products(int i, float* p) const
    {
        if (AL) {
            const uint32_t one = ESZ == 2 ? 0x3f803f80u : 0x3f800000u;
            float s[VEC], r[VEC], w[VEC];
            unpack<ESZ>(*reinterpret_cast<const uint4*>(x + i * ESZ), s);
            unpack<ESZ>(RES ? *reinterpret_cast<const uint4*>(x + residual + i * ESZ) : make_uint4(0, 0, 0, 0), r);
            unpack<ESZ>(g.w ? __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(g.w) + (size_t)i * ESZ))
                            : make_uint4(one, one, one, one), w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) p[e] = (RES ? s[e] + r[e] : s[e]) * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                p[e] = 0.f;
                if (i + e < g.d) {
                    float s = q8_ld1<ESZ>(x, i + e);
                    if (RES) s += q8_ld1<ESZ>(x + residual, i + e);
                    p[e] = s * (g.w ? q8_ld1<ESZ>(g.w, i + e) : 1.f);
                }
            }
        }
    }
};

// Whether a product of the row's part of thread t is not zero, although fp32 may have made
// it so.  The vectors of a padding row are told by their bits.
template <int ESZ, int NV, bool RES, bool AL>
__device__ __forceinline__ bool q8_some_product(const Q8Row<ESZ, RES, AL>& in, int t)
{
    constexpr int VEC = 16 / ESZ;
    constexpr uint32_t digits = ESZ == 2 ? 0x7fff7fffu : 0x7fffffffu;
    bool some = false;
#pragma unroll 1
    for (int j = 0; j < NV; ++j) {
        const int i = in.index(j, t);
        if (i >= in.g.d) break;
        if (AL) {
            const uint4 a = *reinterpret_cast<const uint4*>(in.x + i * ESZ);
            const uint4 b = RES ? *reinterpret_cast<const uint4*>(in.x + in.residual + i * ESZ) : make_uint4(0, 0, 0, 0);
            if (((a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) & digits) == 0u) continue;
        }
#pragma unroll 1
        for (int e = 0; e < VEC && i + e < in.g.d; ++e) some |= in.prod(i + e) != 0.0;
    }
    return some;
}

// Whether a row whose products are all zero in fp32 is one of zeros (padding, as a rule): its
// integers are then written.  Each warp answers for its part, the first, whose thread has
// use for the maximum, for the whole row.  16384 x 4096 bf16 of zeros with a residual: 143 us;
// 1360 by q8_near, which takes every element of a row of tiny values in fp64.
template <int ESZ, int NV, bool RES, bool AL>
__device__ __noinline__ bool q8_zero_row(const Q8RowsArgs& g, const unsigned char* x, int residual, int row)
{
    constexpr int VEC = 16 / ESZ;
    const Q8Row<ESZ, RES, AL> in = {g, x, residual};
    const int tid = threadIdx.x, lane = tid & 31;
    int8_t* qrow = g.q + (size_t)row * g.ldq;
    __syncwarp();  // one warp a row: the other lanes' copies
    int t = tid & ~31;
    const int last = tid < 32 ? (int)blockDim.x - 32 : t;
    for (; t <= last; t += 32)
        if (__any_sync(0xffffffffu, q8_some_product<ESZ, NV, RES, AL>(in, t + lane))) return false;
    for (int j = 0; j < NV; ++j) {
        const int i = in.index(j, tid);
        if (i + VEC <= g.d) {
            if (VEC > 4) *reinterpret_cast<uint2*>(qrow + i) = make_uint2(0u, 0u);
            else *reinterpret_cast<uint32_t*>(qrow + i) = 0u;
        } else {
            for (int e = 0; i + e < g.d; ++e) qrow[i + e] = 0;
        }
    }
    return true;
}

// The values of a warp's part of a row whose rounding fp32 leaves open, decided exactly
// and written again: first 127 |p| against (n + 1/2) max with the fp32 maximum pmf,
// good to 2^-23, which settles most; what that leaves open needs the fp64 maximum, unless
// the products are exact in fp32.  That maximum lies among the values that reach the
// fp32 one to 2^-20, in the parts of the row (s_pm, one a warp) that hold one.  Returns
// the maximum as exactly as it was needed.  Out of line: about one warp in forty comes
// here, and the kernel's registers are its occupancy.
template <int ESZ, int NV, bool RES, bool AL>
__device__ __noinline__ double q8_near(const Q8RowsArgs& g, const unsigned char* x, int residual, int row, float pmf, float k,
                                       const unsigned* s_pm, bool near)
{
    constexpr int VEC = 16 / ESZ;
    const Q8Row<ESZ, RES, AL> in = {g, x, residual};
    const int tid = threadIdx.x, lane = tid & 31, nw = blockDim.x >> 5;
    const bool tiny = pmf < 0x1p-100f, exact = !tiny && !RES && (ESZ == 2 || !g.w);
    int8_t* qrow = g.q + (size_t)row * g.ldq;
    double dm = pmf;
    unsigned todo = 0;  // elements j * VEC + e
    if (near) {
#pragma unroll 1
        for (int j = 0; j < NV; ++j) {
            const int i = in.index(j, tid);
            if (i >= g.d) break;
            float p[VEC];
            in.products(i, p);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float t = p[e] * k;
                if ((AL || i + e < g.d) && (tiny || fabsf(t - rintf(t)) > 0.5f - 0x1p-21f * fabsf(t))) todo |= 1u << (j * VEC + e);
            }
        }
    }
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        unsigned open = 0;
        for (unsigned left = todo; left; left &= left - 1) {
            const int at = __ffs(left) - 1, i = in.index(at / VEC, tid) + at % VEC;
            const double p = in.prod(i);
            if (round == 0 && !exact) {
                const float n = floorf(fabsf((float)p) * k);  // |t| lies within 2^-21 |t| of n + 1/2
                const double diff = fabs(p) * 127.0 - ((double)n + 0.5) * (double)pmf;
                if (tiny || !(fabs(diff) > 0x1p-22 * ((double)n + 0.5) * (double)pmf)) {
                    open |= 1u << at;
                } else {
                    const int m = (int)n + (diff > 0.0 ? 1 : 0);
                    qrow[i] = (int8_t)(p < 0.0 ? -m : m);
                }
            } else {
                qrow[i] = (int8_t)(int)(dm > 0.0 ? rint(p * 127.0 / dm) : 0.0);
            }
        }
        todo = open;
        if (round || !__any_sync(0xffffffffu, todo != 0u)) break;
        const float thr = tiny ? 0.f : pmf * (1.f - 0x1p-20f);
        dm = 0.0;
        __syncwarp();  // one warp a row: the other lanes' copies
        for (int t = 0; t < nw; ++t) {
            if (nw > 1 && !(__uint_as_float(s_pm[t]) >= thr)) continue;
#pragma unroll 1
            for (int j = 0; j < NV; ++j) {
                const int i = in.index(j, 32 * t + lane);
                if (i >= g.d) break;
                float p[VEC];
                in.products(i, p);
                unsigned hit = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) hit |= ((AL || i + e < g.d) && fabsf(p[e]) >= thr ? 1u : 0u) << e;
                for (; hit; hit &= hit - 1) dm = fmax(dm, fabs(in.prod(i + __ffs(hit) - 1)));
            }
        }
        dm = q8_warp_max(dm);
    }
    return dm;
}

constexpr int kQ8RowSlots = 3;

// 16-byte blocks of shared memory for a row of one input (its last vector may reach into
// one block more), and rows of inputs and outputs that a CTA's row needs.
__host__ __device__ constexpr int q8_row_blocks(int nv, int threads) { return nv * threads + 1; }
__host__ __device__ constexpr int q8_rows_kept(bool res, bool al) { return kQ8RowSlots * (res ? 2 : 1) + (al ? 0 : 1); }

// NV vectors of 16 bytes a thread.  blockDim.x threads a row, and blockDim.y rows a CTA
// when blockDim.x is one warp (no barrier then); CTAs walk the rows.
//
// Rows come through shared memory by asynchronous copies, the next row's on the way
// while this one is worked on.  The row's products stay in registers over the
// reduction, two to an instruction throughout.  A warp can be one row ahead of another,
// hence three slots and two sets of partials.
// AL: every row starts on a 16-byte boundary.  Each thread then copies what it reads
// itself, and a row has one barrier.  Otherwise (d * ESZ not a multiple of 16) the
// aligned blocks that hold the row are copied, a vector is read from the two it
// lies in, and out_sum and out_normed are put together in shared memory to leave in
// aligned blocks too (5000 x 4001 bf16 with a residual: 55 us, against 150 us element by
// element).
template <int ESZ, int NV, int MAXT, bool RES, bool AL>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? (NV <= 2 ? 4 : 3) : 1) sv_q8_rows(const __grid_constant__ Q8RowsArgs g)
{
    constexpr int VEC = 16 / ESZ, P = VEC / 2;  // packed pairs of a vector
    constexpr int IN = RES ? 2 : 1;
    extern __shared__ __align__(16) unsigned char q8_rows_dyn[];  // [slots][x, r][rows][blocks], then [rows][blocks] of output
    __shared__ float s_ss[2][32];
    __shared__ unsigned s_pm[2][32];
    __shared__ double s_sd[32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product may load its weights
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nw = nthr >> 5;
    const int stride = gridDim.x * blockDim.y;
    const uint32_t one = ESZ == 2 ? 0x3f803f80u : 0x3f800000u;
    const int RB = q8_row_blocks(NV, nthr), in_step = blockDim.y * RB;  // blocks from an input to the next
    uint4* const slots = reinterpret_cast<uint4*>(q8_rows_dyn) + threadIdx.y * RB;
    uint4* const outs = slots + kQ8RowSlots * IN * in_step;
    const int mine = cdiv_pos(g.d - tid * VEC, nthr * VEC);  // vectors of a row that this thread has (at most NV)
    auto sync_row = [&] {
        if (nw > 1) __syncthreads();
        else __syncwarp();
    };

    auto copy = [&](int row, int slot) {
        const size_t at = (size_t)row * g.d * ESZ;
        const unsigned sh = AL ? 0u : (unsigned)(at & 15u);
        const uint32_t to = lr_smem(slots + slot * IN * in_step + tid);
        const size_t from = at - sh + 16 * (size_t)tid;
        const char* x = static_cast<const char*>(g.x) + from;
        const char* r = RES ? static_cast<const char*>(g.r) + from : nullptr;
        if (AL) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (j >= mine) break;
                q8_cp16(to + 16 * j * nthr, x + 16 * (size_t)(j * nthr), 16);
                if (RES) q8_cp16(to + 16 * (in_step + j * nthr), r + 16 * (size_t)(j * nthr), 16);
            }
        } else {
            // the blocks that hold the row, none of them past the inputs' end
            const int blocks = (int)((sh + (unsigned)g.d * ESZ + 15u) / 16u);
            const size_t end = (size_t)g.M * g.d * ESZ;
#pragma unroll
            for (int j = 0; j <= NV; ++j) {
                if (j * nthr + tid >= blocks) break;
                const int bytes = (int)min((size_t)16, end - from - 16 * (size_t)(j * nthr));
                q8_cp16(to + 16 * j * nthr, x + 16 * (size_t)(j * nthr), bytes);
                if (RES) q8_cp16(to + 16 * (in_step + j * nthr), r + 16 * (size_t)(j * nthr), bytes);
            }
        }
    };
    // a row of output in index order, from shared memory to an unaligned row of global
    auto flush = [&](void* to, size_t at) {
        const unsigned sh = (unsigned)(at & 15u);
        unsigned char* dst = static_cast<unsigned char*>(to) + (at - sh);
        const int bytes = g.d * ESZ, blocks = (int)((sh + (unsigned)bytes + 15u) / 16u);
        for (int b = tid; b < blocks; b += nthr) {
            const int i = 16 * b - (int)sh;  // the row's byte that the block starts with
            if (i >= 0 && i + 16 <= bytes) {
                *reinterpret_cast<uint4*>(dst + 16 * (size_t)b) = sh ? shift16(outs[b - 1], outs[b], 16u - sh) : outs[b];
            } else {
                const unsigned char* src = reinterpret_cast<const unsigned char*>(outs);
                for (int e = 0; e < 16; e += ESZ)
                    if (i + e >= 0 && i + e < bytes) {
                        if (ESZ == 2) *reinterpret_cast<unsigned short*>(dst + 16 * (size_t)b + e) = *reinterpret_cast<const unsigned short*>(src + i + e);
                        else *reinterpret_cast<uint32_t*>(dst + 16 * (size_t)b + e) = *reinterpret_cast<const uint32_t*>(src + i + e);
                    }
            }
        }
    };
    // the weights, as packed as they came
    uint4 wv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        wv[j] = make_uint4(one, one, one, one);
        const int i = (j * nthr + tid) * VEC;
        if (!g.w || j >= mine) continue;
        if (AL || i + VEC <= g.d) {
            wv[j] = __ldg(reinterpret_cast<const uint4*>(g.w) + j * nthr + tid);
        } else {
            float w[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = i + e < g.d ? q8_ld1<ESZ>(g.w, i + e) : 1.f;
            wv[j] = q8_pack<ESZ>(w);
        }
    }
    int row = blockIdx.x * blockDim.y + threadIdx.y, slot = 0, set = 0;
    if (row < g.M) copy(row, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (; row < g.M; row += stride, slot = slot == kQ8RowSlots - 1 ? 0 : slot + 1, set ^= 1) {
        const size_t base = (size_t)row * g.d;
        const unsigned sh = AL ? 0u : (unsigned)(base * ESZ & 15u);
        const uint4* in = slots + slot * IN * in_step;
        const Q8Row<ESZ, RES, AL> in64 = {g, reinterpret_cast<const unsigned char*>(in) + sh, 16 * in_step};
        if (row < g.M - stride) copy(row + stride, slot == kQ8RowSlots - 1 ? 0 : slot + 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (!AL) sync_row();  // the other threads' copies, and the last row's output has left
        unsigned long long p2[NV * P];
        float tm = 0.f, ss;
        {
            unsigned long long acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
            // (the weights stay packed from row to row: unpacked they take twice the registers)
#pragma unroll
            for (int j = 0; j < NV; ++j) asm volatile("" : "+r"(wv[j].x), "+r"(wv[j].y), "+r"(wv[j].z), "+r"(wv[j].w));
            auto get = [&](const uint4* at, int j) {
                if (AL) return at[0];
                uint4 v = shift16(at[0], at[1], sh);
                const int n = (g.d - (j * nthr + tid) * VEC) * ESZ;  // bytes of the row from here on
                if (n < 16) {
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q] = 4 * q >= n ? 0u : (ESZ == 2 && 4 * q + 2 >= n ? w[q] & 0xffffu : w[q]);
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                }
                return v;
            };
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                uint4 x = make_uint4(0, 0, 0, 0), r = x;
                if (j < mine) {
                    x = get(in + j * nthr + tid, j);
                    if (RES) r = get(in + in_step + j * nthr + tid, j);
                }
                unsigned long long a[P], b[P], w[P];
                q8_pairs<ESZ>(x, a);
                if (RES) {
                    q8_pairs<ESZ>(r, b);
#pragma unroll
                    for (int e = 0; e < P; ++e) a[e] = add2(a[e], b[e]);
                }
                q8_pairs<ESZ>(wv[j], w);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    float u, v;
                    acc[j & 1] = fma2(a[e], a[e], acc[j & 1]);
                    p2[j * P + e] = mul2(a[e], w[e]);
                    unpack2(p2[j * P + e], u, v);
                    tm = q8_max3(tm, u, v);
                }
                if (g.sum && j < mine) {  // (may be written over x or r: they are in shared memory)
                    float t[VEC];
#pragma unroll
                    for (int e = 0; e < P; ++e) unpack2(a[e], t[2 * e], t[2 * e + 1]);
                    if (AL) *reinterpret_cast<uint4*>(static_cast<char*>(g.sum) + (base + (size_t)(j * nthr + tid) * VEC) * ESZ) = q8_pack<ESZ>(t);
                    else outs[j * nthr + tid] = q8_pack<ESZ>(t);
                }
            }
            float u, v;
            unpack2(add2(acc[0], acc[1]), u, v);
            ss = u + v;
        }
        // sum s^2 and max |p| (as bits: NaN and inf order above every number)
        unsigned pm = __reduce_max_sync(0xffffffffu, __float_as_uint(tm));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        bool large = !(ss <= 0x1p110f), small = ss < 0x1p-60f && g.eps < 0x1p-60f;
        if (nw > 1) {
            if (lane == 0) { s_ss[set][warp] = ss; s_pm[set][warp] = pm; }
            __syncthreads();
            const float other = lane < nw ? s_ss[set][lane] : 0.f;
            pm = __reduce_max_sync(0xffffffffu, lane < nw ? s_pm[set][lane] : 0u);
            large = __any_sync(0xffffffffu, !(other <= 0x1p110f));
            small = g.eps < 0x1p-60f && __all_sync(0xffffffffu, other < 0x1p-60f);
            if (warp == 0 || g.normed) {
                ss = other;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            }
        }
        if (!AL && g.sum) {
            if (nw == 1) __syncwarp();
            flush(g.sum, base * ESZ);
        }
        const bool bad = pm >= 0x7f800000u;
        const float pmf = __uint_as_float(pm);
        const bool tiny = pmf < 0x1p-100f;  // 127 / pmf, or the products themselves, leave fp32: all in fp64
        // a sum of squares outside fp32's comfortable range is taken again in fp64
        double sd = 0.0;
        const bool again = g.norm && !bad && (large || small);
        if (again) {
#pragma unroll 1
            for (int j = 0; j < NV; ++j)
#pragma unroll 1
                for (int e = 0; e < VEC; ++e)
                    if (in64.index(j, tid) + e < g.d) {
                        const double s = in64.sum(in64.index(j, tid) + e);
                        sd += s * s;
                    }
            sd = q8_warp_sum(sd);
            if (nw > 1) {
                if (lane == 0) s_sd[warp] = sd;
                __syncthreads();
                sd = q8_warp_sum(lane < nw ? s_sd[lane] : 0.0);
                __syncthreads();  // the next row may write s_sd
            }
        }
        // the integers
        const float k = 127.f * __frcp_rn(pmf);
        uint32_t o[NV * P / 2];
        float far = 0.f;  // the largest distance from an integer
        {
            const unsigned long long K2 = pack2(k, k), magic = pack2(0x1.8p23f, 0x1.8p23f);
#pragma unroll
            for (int e = 0; e < NV * P; e += 2) {
                uint32_t lo[2], hi[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // adding 1.5 * 2^23 rounds to an integer, ties to even, in the low bits
                    const unsigned long long t = mul2(p2[e + h], K2), m = add2(t, magic);
                    float u, v;
                    unpack2(sub2(t, sub2(m, magic)), u, v);
                    far = q8_max3(far, u, v);
                    lo[h] = (uint32_t)m;
                    hi[h] = (uint32_t)(m >> 32);
                }
                o[e / 2] = bad ? 0u : __byte_perm(__byte_perm(lo[0], hi[0], 0x0040), __byte_perm(lo[1], hi[1], 0x0040), 0x5410);
            }
        }
        int8_t* qrow = g.q + (size_t)row * g.ldq;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (j * nthr + tid) * VEC;
            if (j >= mine) break;
            if (AL || i + VEC <= g.d) {
                if (VEC > 4) *reinterpret_cast<uint2*>(qrow + i) = make_uint2(o[j * P / 2], o[j * P / 2 + (P > 2 ? 1 : 0)]);
                else *reinterpret_cast<uint32_t*>(qrow + i) = o[j * P / 2];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i + e < g.d) qrow[i + e] = (int8_t)(o[j * P / 2 + e / 4] >> (8 * (e & 3)));
            }
        }
        double ms = 1.0;  // by all where g.normed, else by the first thread
        if (g.norm && (tid == 0 || g.normed)) ms = (again ? sd : (double)ss) / g.d + (double)g.eps;
        if (g.normed) {
            // 1 / rms, or p, leaves fp32; or a p of this thread is subnormal, and its quotient by a
            // small rms would have no more bits than it has
            bool wide = !bad && (tiny || ms < 0x1p-200 || ms > 0x1p200);
            const float inv = bad ? NAN : (ms > 0.0 ? (float)(1.0 / sqrt(ms)) : 0.f);
            if (inv > 1.f) {
                float least = FLT_MIN;
#pragma unroll
                for (int e = 0; e < NV * P; ++e) {
                    const int i = (e / P * nthr + tid) * VEC + 2 * (e % P);
                    float u, v;
                    unpack2(p2[e], u, v);
                    if (AL ? e / P < mine : i < g.d) least = fminf(least, fabsf(u));
                    if (AL ? e / P < mine : i + 1 < g.d) least = fminf(least, fabsf(v));
                }
                wide |= least < FLT_MIN;
            }
            if (!AL && g.sum) sync_row();  // the sums have left
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = (j * nthr + tid) * VEC;
                if (j >= mine) break;
                float y[VEC];
#pragma unroll
                for (int e = 0; e < P; ++e) unpack2(p2[j * P + e], y[2 * e], y[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[e] *= inv;
                if (wide)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const double p = i + e < g.d ? in64.prod(i + e) : 0.0;
                        y[e] = p != 0.0 ? (float)(p / sqrt(ms)) : 0.f;
                    }
                if (AL) *reinterpret_cast<uint4*>(static_cast<char*>(g.normed) + (base + i) * ESZ) = q8_pack<ESZ>(y);
                else outs[j * nthr + tid] = q8_pack<ESZ>(y);
            }
            if (!AL) {
                sync_row();
                flush(g.normed, base * ESZ);
            }
        }
        // values whose rounding fp32 leaves open: seven roundings at most, so within
        // 8 * 2^-24 |t| of a half
        const bool near = !bad && (tiny || far > 0.5f - 0x1p-21f * tm * k);
        double dm = pmf;  // the maximum, as exactly as it is needed
        if (__any_sync(0xffffffffu, near)) {
            if (pm == 0u && q8_zero_row<ESZ, NV, RES, AL>(g, in64.x, in64.residual, row)) dm = 0.0;
            else dm = q8_near<ESZ, NV, RES, AL>(g, in64.x, in64.residual, row, pmf, k, s_pm[set], near);
        }
        if (tid == 0) g.scale[row] = bad ? NAN : (dm > 0.0 ? (float)(dm / (127.0 * sqrt(ms))) : 0.f);
    }
}

// ----------------------------------------------------------------------------- the product

constexpr int kQ8BM = 128;        // channels of a CTA's tile: the MMA's M, or half of it
constexpr int kQ8BK = 128;        // K per block: one 128-byte swizzled row of int8
constexpr int kQ8MaxSub = 2;      // K blocks per stage
constexpr int kQ8MaxNT = 256;     // tokens of an accumulator = the MMA's N
constexpr int kQ8MaxStages = 8;
constexpr int kQ8MaxBufs = 4;     // accumulators in TMEM
constexpr int kQ8EpiWarps = 16;   // per TMEM lane quarter four, on every fourth 16-column chunk
constexpr int kQ8Threads = 128 + 32 * kQ8EpiWarps;
constexpr int kQ8SmemMax = 227 * 1024 - 1024;  // dynamic shared memory of one CTA (static part kept apart)
constexpr int kQ8WBytes = kQ8BM * kQ8BK;

struct Q8GemmArgs {
    void* out;             // [M][V], bf16 or f32
    const float* a_scale;  // [M]
    const float* w_scale;  // [V]
    int* err;              // optional: 1 if a wait gave up
    int M, V, K;
    int nt;                // tokens of an accumulator, a multiple of 16 (pairs: of 32)
    int groups;            // accumulators of a tile (1 or 2): it has groups * nt tokens
    int bufs;              // accumulators in TMEM, `buf_cols` columns each
    int buf_cols, tmem_cols;
    int m_tiles, v_tiles;
    int stages, sub;       // of `sub` K blocks each
    int overlap;           // a programmatic dependent of the kernel that writes a and a_scale
};

// Instruction descriptor: s32 accumulator, signed 8-bit A and B, both K-major, m x n.
__device__ __forceinline__ uint32_t q8_idesc(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void q8_mma(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
            "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
}

// The barrier, in both CTAs of a pair, once this thread's MMAs so far are done.
template <bool PAIR>
__device__ __forceinline__ void q8_commit(uint64_t* bar)
{
    if (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         lr_smem(bar)),
                     "h"((uint16_t)3)
                     : "memory");
    else
        lr_commit(bar);
}

// To this CTA's shared memory; the bytes are counted by `bar`, in a pair the leader's.
template <bool PAIR>
__device__ __forceinline__ void q8_tma(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                lr_smem(dst)),
            "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                lr_smem(dst)),
            "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
            : "memory");
}

// The leader's copy of a shared variable, as a cluster address (this CTA's own without a pair).
template <bool PAIR>
__device__ __forceinline__ uint32_t q8_leader(const void* p)
{
    uint32_t a = lr_smem(p);
    if (PAIR) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(lr_smem(p)));
    return a;
}

__device__ __forceinline__ void q8_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// The producer and the MMA issuer are whole warps in step, one elected lane of which
// issues: addresses, descriptors and loop counts then live in uniform registers, where
// the copies and MMAs want them (from one thread's registers every issue moved its
// operands first).
__device__ __forceinline__ bool q8_elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Wait by a warp, one answer for all lanes: the first look costs one vote.  False (after
// raising the flags) if the phase did not complete within kLrPolls polls, or another
// role of the CTA gave up.
__device__ __forceinline__ bool q8_wait(uint64_t* bar, unsigned parity, volatile int* abort, int* err)
{
    if (__all_sync(0xffffffffu, lr_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, lr_wait(bar, parity, abort, err)) != 0;
}

// A place in a ring and its phase: counted, not divided for.
struct Q8Ring {
    int s = 0;
    unsigned phase = 0;
    __device__ __forceinline__ void next(int S)
    {
        if (++s == S) {
            s = 0;
            phase ^= 1u;
        }
    }
};

// The logits of channel v (one a lane) and the accumulator's tokens m0 .., from TMEM at
// acc: 16-column chunks grp, grp + 4, ...  A bf16 row of even length goes out in words:
// two lanes trade a value, so each stores a channel pair of one of two tokens.
// The tokens' scales may have been written while this kernel was already running (it can
// be a programmatic dependent of the norm), so they are not read as constant memory.
// Three fp32 roundings: the sum, the sum times one scale, that times the other.  A channel's
// scale of at most 1 goes first: the sum times it cannot overflow, and is within a
// rounding of exact down to the least subnormal (an integer times one).  A larger one goes
// last: what overflows before it is beyond fp32's range after it as well.  (The two scales'
// own product may leave the range where the logit does not.)
template <int ESZ>
__device__ __forceinline__ void q8_epilogue(const Q8GemmArgs& g, uint32_t acc, int grp, int m0, int v)
{
    const float sw = v < g.V ? __ldg(g.w_scale + v) : 0.f;
    const unsigned long long sw2 = pack2(sw, sw);
    const bool words = ESZ == 2 && (g.V & 1) == 0;
    const bool wide = (reinterpret_cast<uintptr_t>(g.a_scale) & 15u) == 0;
    const int odd = v & 1;
    const bool sw_first = fabsf(sw) <= 1.f;
    for (int c = grp * 16; c < g.nt && m0 + c < g.M; c += 4 * kQ8EpiWarps) {
        const int left = g.M - (m0 + c);  // tokens from here on
        float sa[16];
        if (wide && left >= 16) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<float4*>(sa + j) = *reinterpret_cast<const float4*>(g.a_scale + m0 + c + j);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) sa[j] = j < left ? g.a_scale[m0 + c + j] : 0.f;
        }
        uint32_t r[16];
        q8_tmem_ld16(acc + (uint32_t)c, r);
        float z[16];
        if (__all_sync(0xffffffffu, sw_first)) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const unsigned long long p = pack2((float)(int)r[j], (float)(int)r[j + 1]);
                unpack2(mul2(mul2(p, sw2), pack2(sa[j], sa[j + 1])), z[j], z[j + 1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = (float)(int)r[j] * (sw_first ? sw : sa[j]) * (sw_first ? sa[j] : sw);
        }
        const bool in = v < g.V;  // (the others still take part in the loads and the trade)
        if (words) {
            uint32_t* to = static_cast<uint32_t*>(g.out) + ((size_t)(m0 + c + odd) * g.V + (v - odd)) / 2;
            const size_t step = (size_t)g.V;  // words of two rows
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float other = __shfl_xor_sync(0xffffffffu, odd ? z[j] : z[j + 1], 1);
                const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(other, z[j + 1]) : __floats2bfloat162_rn(z[j], other);
                if (j + odd < left && in) *to = *reinterpret_cast<const uint32_t*>(&h);
                to += step;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < left && in) q8_st1<ESZ>(g.out, (size_t)(m0 + c + j) * g.V + v, z[j]);
        }
    }
}

// Persistent, one CTA per SM, or a pair of them (PAIR: cta_group::2) on one tile of 256
// channels: each CTA holds its 128 channels and HALF the tokens, and gets all of the
// tile's columns for its channels, so an SM's shared memory is filled and read with two
// thirds of the bytes a product.  The pair's leader waits, issues and commits for both.
// Tiles are walked with the token tile fastest, so those that share weights run at about
// the same time.  A tile of two accumulators (groups = 2) reads its weights once for both.
// Every wait on an mbarrier is bounded: past kLrPolls polls the CTA raises *err, stops
// issuing, and still frees its TMEM.
template <int ESZ, bool PAIR>
__global__ void __launch_bounds__(kQ8Threads, 1)
    sv_q8_gemm(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ta, Q8GemmArgs g)
{
    extern __shared__ unsigned char q8_dyn[];
    // every block on a 1024-byte boundary of the shared window (the swizzle atom)
    unsigned char* ring = q8_dyn + ((1024u - (lr_smem(q8_dyn) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t full[kQ8MaxStages], empty[kQ8MaxStages], tfull[kQ8MaxBufs], tempty[kQ8MaxBufs];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;

    constexpr int CTAS = PAIR ? 2 : 1;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    int rank = 0;
    if (PAIR) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int kbs = (g.K + kQ8BK - 1) / kQ8BK, S = g.stages, G = g.groups;
    const int mine = g.nt / CTAS, a_bytes = mine * kQ8BK;  // this CTA's tokens of an accumulator
    const int BLOCK = kQ8WBytes + G * a_bytes, SUB = g.sub, STAGE = SUB * BLOCK;
    const unsigned tiles = (unsigned)g.m_tiles * (unsigned)g.v_tiles, m_tiles = (unsigned)g.m_tiles;  // fits an int
    const unsigned first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            lr_mbar_init(&full[s], 1);
            lr_mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < g.bufs; ++b) {
            lr_mbar_init(&tfull[b], 1);
            lr_mbar_init(&tempty[b], CTAS * kQ8EpiWarps);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(lr_smem(&s_tmem)),
                         "r"(g.tmem_cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(lr_smem(&s_tmem)),
                         "r"(g.tmem_cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    lr_fence_before();
    __syncthreads();
    if (PAIR) q8_cluster_sync();  // both CTAs' barriers stand before either is reached from the other
    lr_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* abort = &s_abort;

    if (warp == 0) {
        // ---- producer of this CTA's share of every stage
        Q8Ring r;
        int it = 0;
        bool ok = true;
        const uint32_t bars = q8_leader<PAIR>(full);
        // a place among the stages to load: K block kb of tile t, whose rows start at m0 and v0
        struct Place {
            unsigned t;
            int kb, m0, v0;
        };
        auto tile = [&](Place& p) {
            p.kb = 0;
            const unsigned v = p.t / m_tiles;
            p.m0 = (int)(p.t - v * m_tiles) * G * g.nt + rank * mine;
            p.v0 = ((int)v * CTAS + rank) * kQ8BM;
        };
        auto next = [&](Place& p) {
            if ((p.kb += SUB) >= kbs) {
                p.t += step;
                tile(p);
            }
        };
        // the weights' and / or the tokens' copies of a stage, into place s of the ring
        auto issue = [&](const Place& p, int s, bool weights, bool tokens) {
            if (q8_elect()) {
                unsigned char* st = ring + s * STAGE;
                const uint32_t bar = bars + 8u * s;
                const int subs = min(SUB, kbs - p.kb);
                if (weights && rank == 0) lr_expect_tx(&full[s], (unsigned)(CTAS * subs * BLOCK));
                for (int u = 0; u < subs; ++u, st += BLOCK) {
                    const int x = (p.kb + u) * kQ8BK;
                    if (weights) q8_tma<PAIR>(st, &tw, bar, x, p.v0);
                    if (tokens) q8_tma<PAIR>(st + kQ8WBytes, &ta, bar, x, p.m0);
                    if (tokens && G > 1) q8_tma<PAIR>(st + kQ8WBytes + a_bytes, &ta, bar, x, p.m0 + g.nt);
                }
            }
            __syncwarp();
        };
        // the first round of the ring; where the kernel before is the norm of the tokens, the
        // weights do not wait for it
        Place p = {first, 0, 0, 0};
        tile(p);
        Place p0 = p;
        if (g.overlap) {
            for (; it < S && p.t < tiles; ++it, next(p)) issue(p, it, true, false);
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int u = 0; u < it; ++u, next(p0)) issue(p0, u, false, true);
        } else {
            for (; it < S && p.t < tiles; ++it, next(p)) issue(p, it, true, true);
        }
        if (it == S) r.phase = 1u;
        for (; p.t < tiles; ++it, next(p)) {
            ok = q8_wait(&empty[r.s], r.phase ^ 1u, abort, g.err);
            if (!ok) break;
            issue(p, r.s, true, true);
            r.next(S);
        }
        // every stage handed back: nothing of the pair's is still on its way to this CTA
        for (int u = max(0, it - S); ok && u < it; ++u) ok = q8_wait(&empty[u % S], (unsigned)(u / S) & 1u, abort, g.err);
    } else if (warp == 1 && rank == 0) {
        // ---- MMA issuer
        const uint32_t idesc = q8_idesc(CTAS * kQ8BM, g.nt);
        const uint64_t w0 = lr_desc(lr_smem(ring)), a_off = kQ8WBytes >> 4, g_off = (uint64_t)(a_bytes >> 4);
        Q8Ring r, acc;
        int used = 0;  // accumulators so far, up to g.bufs
        bool ok = true;
        // the products of stage place s, K blocks kb .., into accumulators h0 .. h1
        uint32_t d[2];
        auto products = [&](int s, int kb, int h0, int h1) {
            uint64_t w = w0 + (uint64_t)((unsigned)(s * STAGE) >> 4);
#pragma unroll
            for (int u = 0; u < kQ8MaxSub; ++u, w += (unsigned)BLOCK >> 4) {
                if (u >= SUB || kb + u >= kbs) break;
#pragma unroll
                for (int j = 0; j < kQ8BK / 32; ++j) {  // K = 32 per MMA: 32 bytes along the swizzled row
                    const uint32_t on = (kb + u > 0 || j > 0) ? 1u : 0u;
                    if (h0 == 0) q8_mma<PAIR>(d[0], w + 2 * j, w + a_off + 2 * j, idesc, on);
                    if (h1 == 1) q8_mma<PAIR>(d[1], w + 2 * j, w + a_off + g_off + 2 * j, idesc, on);
                }
            }
        };
        for (unsigned t = first; ok && t < tiles; t += step) {
            int buf[2];
            unsigned parity[2];
            bool taken[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h >= G) break;
                buf[h] = acc.s;
                parity[h] = acc.phase ^ 1u;
                taken[h] = used >= g.bufs;
                d[h] = tmem + (uint32_t)(acc.s * g.buf_cols);
                used += taken[h] ? 0 : 1;
                acc.next(g.bufs);
            }
            if (taken[0] && !q8_wait(&tempty[buf[0]], parity[0], abort, g.err)) { ok = false; break; }
            lr_fence_after();
            // while the second accumulator is still being stored, the first goes ahead through
            // the stages of the ring (a look that may not sleep until it is stored: 300 x 768 x
            // 69001 bf16 38.9 us, 39.6 by a wait that may, 39.1 without going ahead)
            int ahead = 0;
            if (G > 1 && taken[1] && !__all_sync(0xffffffffu, lr_test(&tempty[buf[1]], parity[1]))) {
                Q8Ring p = r;
                for (int kb = 0; kb < kbs && ahead < S; kb += SUB, ++ahead) {
                    ok = q8_wait(&full[p.s], p.phase, abort, g.err);
                    if (!ok) break;
                    lr_fence_after();
                    if (q8_elect()) products(p.s, kb, 0, 0);
                    __syncwarp();
                    p.next(S);
                }
                ok = ok && q8_wait(&tempty[buf[1]], parity[1], abort, g.err);
            }
            if (!ok) break;
            lr_fence_after();
            for (int kb = 0, n = 0; kb < kbs; kb += SUB, ++n) {
                if (n >= ahead && !q8_wait(&full[r.s], r.phase, abort, g.err)) { ok = false; break; }
                lr_fence_after();
                if (q8_elect()) {
                    products(r.s, kb, n >= ahead ? 0 : 1, G - 1);
                    q8_commit<PAIR>(&empty[r.s]);
                }
                __syncwarp();
                r.next(S);
            }
            if (ok && q8_elect()) {
                q8_commit<PAIR>(&tfull[buf[0]]);
                if (G > 1) q8_commit<PAIR>(&tfull[buf[1]]);
            }
            __syncwarp();
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp 4 + e owns TMEM lanes (= this CTA's channels) 32q .. 32q + 31,
        // q = e % 4, and the 16-column chunks e / 4, e / 4 + 4, ...
        const int q = (warp - 4) & 3, grp = (warp - 4) >> 2;
        Q8Ring acc;
        bool ok = true;
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the tokens' scales
        for (unsigned t = first; ok && t < tiles; t += step) {
            const unsigned vt = t / m_tiles;
            const int m0 = (int)(t - vt * m_tiles) * G * g.nt;
            const int v = ((int)vt * CTAS + rank) * kQ8BM + 32 * q + lane;
            for (int h = 0; h < G; ++h) {
                // the warp-wide tcgen05.ld below runs on all lanes or none
                ok = q8_wait(&tfull[acc.s], acc.phase, abort, g.err);
                if (!ok) break;
                lr_fence_after();
                q8_epilogue<ESZ>(g, tmem + (uint32_t)(acc.s * g.buf_cols) + ((uint32_t)(32 * q) << 16), grp, m0 + h * g.nt, v);
                lr_fence_before();
                __syncwarp();
                if (lane == 0)
                    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(q8_leader<PAIR>(&tempty[acc.s]))
                                 : "memory");
                acc.next(g.bufs);
            }
        }
    }
    __syncwarp();
    // after a wait gave up: time for the copies in flight to land before the memory goes
    // away (two milliseconds, a thousand times what one takes)
    if (threadIdx.x == 0 && s_abort) {
        uint64_t t0, t1;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        for (unsigned k = 0; k < kLrPolls; ++k) {
            asm volatile("nanosleep.u32 1000;");
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
            if (t1 - t0 > 2000000u) break;
        }
    }
    lr_fence_before();
    __syncthreads();
    if (PAIR) q8_cluster_sync();  // neither CTA leaves while the other may still reach its barriers
    if (warp == 2) {
        lr_fence_after();
        if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_cols));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.tmem_cols));
    }
}

}  // namespace sv
