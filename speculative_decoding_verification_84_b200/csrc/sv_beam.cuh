// sv_beam.cuh -- growing a draft tree by beams [SpecLA, Metodologia 1: drafts shaped
// as branching trees; Metodologia 3: paths ranked by cumulative draft
// log-probability]: the selection of a level's K nodes over beams and vocabulary,
// and the draft's states following them.
//
// The selection.  Candidate (w, v) of a sequence has the key
//     score[w] + l[w][v] / T - lse(l[w] / T);
// the K largest keys win, ties to the lower beam, then the lower token.  Inside a
// beam the keys order as the logits do, whatever its normaliser, so ONE pass over
// the logits gives both what the normaliser needs and the beam's best K logits:
//   sv_beam_rows   one CTA per (row, segment): the segment in registers, each
//                  warp's (offset, sum of exponentials), and the segment's best K
//                  logits in order.  The K-th largest of the 32 maxima of groups
//                  of 8 lanes bounds the K-th largest logit from below, so the
//                  few elements at or above it (about K of them) are collected
//                  and ranked by counting; if ties make them many, the K best are
//                  taken one by one.
//   sv_beam_merge  one CTA per sequence, a warp per beam: the row's normaliser in
//                  fp64, its K best from the segments' sorted lists by K rounds of
//                  a warp-wide maximum over the lists' heads; then one warp, a lane
//                  per beam, takes the K best keys (fp64) the same way.  A
//                  programmatic dependent of sv_beam_rows.
// Segments are cut by token index, so equal rows give equal normalisers wherever
// they lie in memory.
//
// The states.  sv_beam_reorder copies dst[l][b][k] = src[l][b][parent[b][k]], the
// live tokens of each, every source vector loaded once for all children of a parent.
#pragma once

#include "sv_common.cuh"

namespace sv {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMaxNV = 8;       // 16-byte vectors per thread
constexpr int kBeamMaxSegs = 128;   // segments per row (4 lists per lane of the merge)
constexpr int kBeamCap = 512;       // collected candidates of a segment

struct BeamArgs {
    const void* logits;        // [B][W][V]
    const float* score;        // [B][W]
    const float* temperature;  // [B]
    const int32_t* frozen;     // [B][W] or null
    float4* part;              // [B*W][nseg][kBeamWarps] (m, mk, s, 0)
    uint2* list;               // [B*W][nseg][K] (logit bits, token), best first
    int32_t* out_parent;       // [B][K]
    int32_t* out_token;        // [B][K]
    float* out_score;          // [B][K]
    int32_t* out_status;       // [B] or null
    int B, W, V, K, nseg, seg;  // seg: tokens per segment, a multiple of the vector
    int pad_token;
};

__device__ __forceinline__ bool beam_t_ok(float T) { return T == 0.f || (T >= SV_TEMPERATURE_MIN && T <= FLT_MAX); }

// A 16-byte vector of row elements [i, i + VEC) of a row that may start off a 16-byte
// boundary; elements past V are -inf.  Reads only 16-byte blocks that hold a wanted
// element, and no byte past `end`.
template <int ESZ>
__device__ __forceinline__ uint4 beam_ld(const unsigned char* row, int i, int V, const unsigned char* end)
{
    constexpr int VEC = 16 / ESZ;
    const unsigned char* p = row + (size_t)i * ESZ;
    const unsigned sh = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
    if (sh == 0 && i + VEC <= V) return ld_stream(reinterpret_cast<const uint4*>(p));
    if (i + VEC <= V && p - sh + 32 <= end) {
        const uint4* a = reinterpret_cast<const uint4*>(p - sh);
        const uint4 lo = __ldg(a), hi = __ldg(a + 1);
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const unsigned b = (sh & 3u) * 8u;
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // sh / 4 whole words, then sh % 4 bytes (sh is one value for the row)
            const uint32_t a0 = sh < 4 ? w[k] : (sh < 8 ? w[k + 1] : (sh < 12 ? w[k + 2] : w[k + 3]));
            const uint32_t a1 = sh < 4 ? w[k + 1] : (sh < 8 ? w[k + 2] : (sh < 12 ? w[k + 3] : w[(k + 4) & 7]));
            o[k] = __funnelshift_r(a0, a1, b);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (ESZ == 4) {
            o[k] = i + k < V ? __ldg(reinterpret_cast<const uint32_t*>(p) + k) : 0xff800000u;
        } else {
            const uint32_t a = i + 2 * k < V ? __ldg(reinterpret_cast<const unsigned short*>(p) + 2 * k) : 0xff80u;
            const uint32_t b = i + 2 * k + 1 < V ? __ldg(reinterpret_cast<const unsigned short*>(p) + 2 * k + 1) : 0xff80u;
            o[k] = a | b << 16;
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// (value, index) ranks before: larger value, then smaller index
__device__ __forceinline__ bool beam_before(float av, int ai, float bv, int bi) { return av > bv || (av == bv && ai < bi); }

// Floats as integers of the same order (-0 first made +0).
__device__ __forceinline__ unsigned beam_ord(float v)
{
    const unsigned u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

template <int ESZ, int NV>
__global__ void __launch_bounds__(kBeamThreads) sv_beam_rows(BeamArgs g)
{
    constexpr int VEC = 16 / ESZ;
    __shared__ float s_group[32];
    __shared__ float s_v[kBeamCap];
    __shared__ int s_i[kBeamCap];
    __shared__ float s_tau;
    __shared__ int s_n;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x / g.nseg, seg = blockIdx.x % g.nseg, b = row / g.W;
    const float T = __ldg(g.temperature + b), sc = __ldg(g.score + row);
    // no candidate comes from this row's logits
    if (!beam_t_ok(T) || !(sc > -INFINITY && sc < INFINITY) || (g.frozen && __ldg(g.frozen + row))) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned char* base = static_cast<const unsigned char*>(g.logits);
    const unsigned char* end = base + (size_t)g.B * g.W * g.V * ESZ;
    const unsigned char* rp = base + (size_t)row * g.V * ESZ;
    const int i0 = seg * g.seg, i1 = min(g.V, i0 + g.seg);

    uint4 v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = i0 + (j * kBeamThreads + tid) * VEC;
        const uint32_t ninf = ESZ == 2 ? 0xff80ff80u : 0xff800000u;
        v[j] = i < i1 ? beam_ld<ESZ>(rp, i, g.V, end) : make_uint4(ninf, ninf, ninf, ninf);
    }
    float m = vec_max<ESZ>(v[0]);
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, vec_max<ESZ>(v[j]));
    const float tmax = m;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((lane & 7) == 0) s_group[warp * 4 + (lane >> 3)] = m == m ? m : -INFINITY;
    if (tid == 0) s_n = 0;
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // the warp's exponentials against its own integer offset (T = 0 needs the NaN test only)
    {
        float khi = 1.f, klo = 0x1p-60f;
        if (T > 0.f) split_k(T, &khi, &klo);
        // (kept finite where a warp holds only the type's lowest values: its sum is then 0)
        const float mk = m == -INFINITY ? 0.f : fmaxf(ceilf(__fmul_rn(m, khi)), -3e38f);
        unsigned long long acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = pack2(0.f, 0.f);
        lazy_exps_add<ESZ, NV>(acc, v, khi, klo, mk);
        const float s = lazy_warp_sum(acc);
        if (lane == 0) g.part[((size_t)row * g.nseg + seg) * kBeamWarps + warp] = make_float4(m, mk, s, 0.f);
    }
    __syncthreads();
    if (warp == 0) {
        // the K-th largest of the 32 group maxima
        const float x = s_group[lane];
        int rank = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float y = __shfl_sync(0xffffffffu, x, j);
            rank += (y > x || (y == x && j < lane)) ? 1 : 0;
        }
        if (rank == g.K - 1) s_tau = x;
    }
    __syncthreads();
    const float tau = s_tau;
    if (tmax >= tau) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[VEC];
            unpack<ESZ>(v[j], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if (x[e] >= tau && x[e] > -INFINITY) {
                    const int at = atomicAdd(&s_n, 1);
                    if (at < kBeamCap) {
                        s_v[at] = x[e];
                        s_i[at] = i0 + (j * kBeamThreads + tid) * VEC + e;
                    }
                }
            }
        }
    }
    __syncthreads();
    const int n = s_n;
    uint2* list = g.list + ((size_t)row * g.nseg + seg) * g.K;
    if (n <= kBeamCap) {
        for (int c = tid; c < n; c += kBeamThreads) {
            const float x = s_v[c];
            const int i = s_i[c];
            int rank = 0;
            for (int o = 0; o < n; ++o) rank += beam_before(s_v[o], s_i[o], x, i) ? 1 : 0;
            if (rank < g.K) list[rank] = make_uint2(__float_as_uint(x), (unsigned)i);
        }
        for (int c = n + tid; c < g.K; c += kBeamThreads) list[c] = make_uint2(0xff800000u, 0xffffffffu);
        return;
    }
    // many equal logits at the border: the best one after the last taken, K times
    float lv = INFINITY;
    int li = -1;
    for (int k = 0; k < g.K; ++k) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[VEC];
            unpack<ESZ>(v[j], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = i0 + (j * kBeamThreads + tid) * VEC + e;
                if (beam_before(lv, li, x[e], i) && beam_before(x[e], i, bv, bi) && x[e] > -INFINITY) { bv = x[e]; bi = i; }
            }
        }
        const unsigned o = beam_ord(bv), top = __reduce_max_sync(0xffffffffu, o);
        const unsigned mi = __reduce_min_sync(0xffffffffu, o == top ? (unsigned)bi : 0x7fffffffu);
        if (o == top && (unsigned)bi == mi) { s_v[warp] = bv; s_i[warp] = bi; }
        __syncthreads();
        bv = s_v[0];
        bi = s_i[0];
        for (int w = 1; w < kBeamWarps; ++w)
            if (beam_before(s_v[w], s_i[w], bv, bi)) { bv = s_v[w]; bi = s_i[w]; }
        __syncthreads();
        lv = bv;
        li = bi;
        if (tid == 0) list[k] = make_uint2(__float_as_uint(bv), bv > -INFINITY ? (unsigned)bi : 0xffffffffu);
    }
}

// 32 W threads: warp w merges beam w.  Dynamic shared memory: W x K pairs.
__global__ void __launch_bounds__(1024) sv_beam_merge(BeamArgs g)
{
    extern __shared__ __align__(8) unsigned char beam_dyn[];
    double* s_key = reinterpret_cast<double*>(beam_dyn);         // [W][K]
    int* s_tok = reinterpret_cast<int*>(s_key + g.W * g.K);      // [W][K]
    int* s_cnt = s_tok + g.W * g.K;                              // [W]
    int* s_bad = s_cnt + g.W;                                    // [W]
    const int b = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const size_t row = (size_t)b * g.W + w;
    const float T = __ldg(g.temperature + b), sc = __ldg(g.score + row);
    const bool frozen = g.frozen && __ldg(g.frozen + row);
    const bool t_ok = beam_t_ok(T);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int cnt = 0, bad = 0;
    if (!(sc < INFINITY)) {
        bad = SV_ROW_BAD_SCORE;
    } else if (sc == -INFINITY) {
    } else if (frozen) {
        cnt = 1;
        if (lane == 0) { s_key[w * g.K] = (double)sc; s_tok[w * g.K] = g.pad_token; }
    } else if (t_ok) {
        // the row's normaliser
        float M_ = -INFINITY, MK = 0.f;
        double S = 0.0;
        int nan = 0;
        const float4* part = g.part + row * g.nseg * kBeamWarps;
        for (int t = lane; t < g.nseg * kBeamWarps; t += 32) {
            const float4 p = part[t];
            nan |= (p.z != p.z);
            if (p.x == -INFINITY) continue;
            if (M_ == -INFINITY) { M_ = p.x; MK = p.y; S = (double)p.z; continue; }
            if (p.y > MK) { S = S * pow2d(MK - p.y) + (double)p.z; MK = p.y; }
            else S += (double)p.z * pow2d(p.y - MK);
            M_ = fmaxf(M_, p.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, M_, o);
            const float mk2 = __shfl_xor_sync(0xffffffffu, MK, o);
            const double s2 = __shfl_xor_sync(0xffffffffu, S, o);
            nan |= __shfl_xor_sync(0xffffffffu, nan, o);
            if (m2 == -INFINITY) continue;
            if (M_ == -INFINITY) { M_ = m2; MK = mk2; S = s2; continue; }
            if (mk2 > MK) { S = S * pow2d(MK - mk2) + s2; MK = mk2; }
            else S += s2 * pow2d(mk2 - MK);
            M_ = fmaxf(M_, m2);
        }
        if (nan || M_ == -INFINITY || M_ == INFINITY || (T > 0.f && !(S > 0.0 && S <= DBL_MAX && MK <= FLT_MAX))) {
            bad = SV_ROW_BAD_LOGITS;
        } else {
            const double lse = T > 0.f ? ((double)MK + log2(S)) * kLn2 : 0.0;
            const int want = T > 0.f ? g.K : 1;  // T = 0: all mass on the first argmax
            const uint2* list = g.list + row * g.nseg * g.K;
            constexpr int LL = kBeamMaxSegs / 32;  // lists per lane
            int at[LL];
            unsigned hv[LL], hi[LL];
#pragma unroll
            for (int l = 0; l < LL; ++l) {
                const int s = l * 32 + lane;
                at[l] = 0;
                hv[l] = 0u;  // below every number's order
                hi[l] = 0xffffffffu;
                if (s < g.nseg) {
                    const uint2 h = list[(size_t)s * g.K];
                    if (h.y != 0xffffffffu) { hv[l] = beam_ord(__uint_as_float(h.x)); hi[l] = h.y; }
                }
            }
            for (int k = 0; k < want; ++k) {
                unsigned bv = hv[0], bi = hi[0];
#pragma unroll
                for (int l = 1; l < LL; ++l)
                    if (hv[l] > bv || (hv[l] == bv && hi[l] < bi)) { bv = hv[l]; bi = hi[l]; }
                const unsigned top = __reduce_max_sync(0xffffffffu, bv);
                if (top == 0u) break;
                const unsigned ti = __reduce_min_sync(0xffffffffu, bv == top ? bi : 0xffffffffu);
                if (bv == top && bi == ti) {
                    const unsigned u = top ^ ((top >> 31) ? 0x80000000u : 0xffffffffu);
                    const double l = (double)__uint_as_float(u);
                    s_key[w * g.K + k] = T > 0.f ? (double)sc + (l / (double)T - lse) : (double)sc;
                    s_tok[w * g.K + k] = (int)ti;
#pragma unroll
                    for (int q = 0; q < LL; ++q) {
                        if (hi[q] == ti) {
                            hv[q] = 0u;
                            hi[q] = 0xffffffffu;
                            if (++at[q] < g.K) {
                                const uint2 h = list[(size_t)(q * 32 + lane) * g.K + at[q]];
                                if (h.y != 0xffffffffu) { hv[q] = beam_ord(__uint_as_float(h.x)); hi[q] = h.y; }
                            }
                        }
                    }
                }
                ++cnt;
            }
        }
    }
    if (lane == 0) { s_cnt[w] = cnt; s_bad[w] = bad; }
    __syncthreads();
    if (w != 0) return;
    // a lane per beam: the K best keys, ties to the lower beam
    const int have = lane < g.W ? s_cnt[lane] : 0;
    int p = 0;
    for (int k = 0; k < g.K; ++k) {
        unsigned long long o = 0ull;
        double key = -INFINITY;
        if (p < have) {
            key = s_key[lane * g.K + p] + 0.0;
            const unsigned long long u = (unsigned long long)__double_as_longlong(key);
            o = u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
        }
        const unsigned hi = (unsigned)(o >> 32), th = __reduce_max_sync(0xffffffffu, hi);
        const unsigned lo = hi == th ? (unsigned)o : 0u, tl = __reduce_max_sync(0xffffffffu, lo);
        const unsigned who = __ballot_sync(0xffffffffu, p < have && hi == th && (unsigned)o == tl);
        const size_t at = (size_t)b * g.K + k;
        if (who == 0u) {
            if (lane == 0) { g.out_parent[at] = -1; g.out_token[at] = -1; g.out_score[at] = -INFINITY; }
        } else if (lane == __ffs(who) - 1) {
            g.out_parent[at] = lane;
            g.out_token[at] = s_tok[lane * g.K + p];
            g.out_score[at] = (float)key;
            ++p;
        }
    }
    if (g.out_status) {
        int st = __reduce_or_sync(0xffffffffu, lane < g.W ? (unsigned)s_bad[lane] : 0u);
        if (!t_ok) st |= SV_ROW_BAD_TEMPERATURE;
        if (lane == 0) g.out_status[b] = st;
    }
}

// ----------------------------------------------------------------------------- states

struct ReorderArgs {
    const unsigned char* src;  // [L][B][W][H][S][tb]
    unsigned char* dst;        // [L][B][K][H][S][tb]
    const int32_t* parent;     // [B][K]
    const int32_t* lengths;    // [B] or null (S)
    long long S, tb;           // tokens of a block, bytes of a token
    long long chunks;          // L B H
    int B, W, K, H;
    int tx;                    // threads along a block (a power of two, 8 .. 256)
};

constexpr int kReorderThreads = 256;
constexpr int kReorderU = 4;  // vectors per thread and source

// VT: the widest access that divides token and block sizes and the base addresses.
template <class VT>
__global__ void __launch_bounds__(kReorderThreads) sv_beam_reorder(ReorderArgs g)
{
    // a CTA: 256 / tx blocks (l, b, h) x tx * kReorderU vectors of each
    __shared__ int s_parent[kReorderThreads / 8][SV_MAX_BEAMS];
    __shared__ unsigned s_same[kReorderThreads / 8][SV_MAX_BEAMS];
    const int ty = kReorderThreads / g.tx, y = threadIdx.x / g.tx, x = threadIdx.x % g.tx;
    const long long vecs = g.S * g.tb / (long long)sizeof(VT);
    const long long tiles = (vecs + (long long)g.tx * kReorderU - 1) / ((long long)g.tx * kReorderU);
    const long long c0 = (blockIdx.x / tiles) * ty, tile = blockIdx.x % tiles;
    for (int e = threadIdx.x; e < ty * g.K; e += kReorderThreads) {
        const long long c = c0 + e / g.K;
        const int b = (int)((c / g.H) % g.B), k = e % g.K;
        int p = -1;
        if (c < g.chunks) p = g.parent[(size_t)b * g.K + k];
        s_parent[e / g.K][k] = (p >= 0 && p < g.W) ? p : -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < ty * g.K; e += kReorderThreads) {
        const int yy = e / g.K, k = e % g.K, p = s_parent[yy][k];
        unsigned same = 0;  // the children of p, at its first one
        if (p >= 0) {
            bool first = true;
            for (int o = 0; o < g.K; ++o)
                if (s_parent[yy][o] == p) {
                    if (o < k) first = false;
                    same |= 1u << o;
                }
            if (!first) same = 0;
        }
        s_same[yy][k] = same;
    }
    __syncthreads();
    const long long c = c0 + y;
    if (c >= g.chunks) return;
    const int h = (int)(c % g.H), b = (int)((c / g.H) % g.B);
    const long long l = c / ((long long)g.H * g.B);
    long long live = g.S;
    if (g.lengths) live = min(g.S, max(0ll, (long long)g.lengths[b]));
    const long long n = live * g.tb / (long long)sizeof(VT);
    const long long i0 = tile * g.tx * kReorderU + x;
    if (i0 >= n) return;
    const VT* src = reinterpret_cast<const VT*>(g.src) + ((l * g.B + b) * g.W * g.H + h) * vecs;
    VT* dst = reinterpret_cast<VT*>(g.dst) + ((l * g.B + b) * g.K * g.H + h) * vecs;
    for (int k = 0; k < g.K; ++k) {
        unsigned same = s_same[y][k];
        if (!same) continue;
        const VT* from = src + (long long)s_parent[y][k] * g.H * vecs;
        VT v[kReorderU];
#pragma unroll
        for (int u = 0; u < kReorderU; ++u)
            if (i0 + u * g.tx < n) v[u] = __ldg(from + i0 + u * g.tx);
        while (same) {
            const int kk = __ffs(same) - 1;
            same &= same - 1;
            VT* to = dst + (long long)kk * g.H * vecs;
#pragma unroll
            for (int u = 0; u < kReorderU; ++u)
                if (i0 + u * g.tx < n) to[i0 + u * g.tx] = v[u];
        }
    }
}

}  // namespace sv
