// sv_beam.cuh -- growing a draft tree by beams [SpecLA, Metodologia 1: drafts shaped
// as branching trees; Metodologia 3: paths ranked by cumulative draft
// log-probability]: the selection of a level's K nodes over beams and vocabulary,
// and the draft's states following them.
//
// The selection.  Candidate (w, v) of a sequence has the key
//     score[w] + l[w][v] / T - lse(l[w] / T);
// the K largest keys win, ties to the lower beam, then the lower token.  Inside a
// beam the keys order as the logits do, whatever its normaliser, and a row's K
// best logits lie in the K chunks of largest maximum (ties: the earlier chunk, which
// holds the smaller tokens).  So the pass over the logits selects nothing:
//   sv_beam_rows   every warp walks a span of the rows: per batch of 8 vectors a
//                  lane (offset, sum of exponentials), per chunk (L lanes of one
//                  vector) its maximum.  No barrier.
//   sv_beam_pick   one CTA per row: the normaliser in fp64; the K best chunks, of
//                  which it reads the logits again (K L vectors, from L2); the
//                  logits at or above the K-th chunk's maximum (about K), ranked
//                  by counting.  The sequence's first CTA (or the last to finish)
//                  places the beams' candidates by their keys (fp64) the same way.
//                  A programmatic dependent of sv_beam_rows.
// Selecting inside the pass (each CTA its segment's K best, with group maxima for a
// threshold) cost more than the pass does: 64 x 8 x 128256 bf16, K = 8, took 96 us in
// that form and 46 when first parted; now 37.8, of which the pass is 27.
// Rows of many equal logits (all of them, say) leave the counting for one look a pick:
// 66 us of that shape flat, 329 with K = 32 (54 otherwise).  A row that counts for nothing
// is not read, but its warps have nothing else to do: a first level of that shape, one
// live beam of eight, takes 26 us.
// Batches are cut by token index, so equal rows give equal normalisers wherever
// they lie in memory.
//
// The states.  sv_beam_reorder copies dst[l][b][k] = src[l][b][parent[b][k]], the
// live tokens of each, every source vector loaded once for all children of a parent.
#pragma once

#include "sv_common.cuh"

namespace sv {

constexpr int kBeamThreads = 256;
constexpr int kBeamNV = 8;          // vectors a lane and batch
constexpr int kPickThreads = 128;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickCluster = 8;     // the most rows of a sequence that are one cluster
constexpr int kBeamCap = 1024;      // candidates of a row, and a sequence's W K keys
constexpr int kPickChunks = 64;     // chunks a row is looked for in without choosing among them

struct BeamArgs {
    const void* logits;        // [B][W][V]
    const float* score;        // [B][W]
    const float* temperature;  // [B]
    const int32_t* frozen;     // [B][W] or null
    float2* part;              // [B*W][nb] (max, sum) of each batch
    float* cmax;               // [B*W][nch] chunk maxima, nch = nb * 4 * (32 / L)
    double* key;               // [B*W][K] each row's candidates' keys, best first
    int32_t* tok;              // [B*W][K] and tokens
    int2* row_info;            // [B*W] (candidates, status bits)
    unsigned* ticket;          // [B] rows finished
    int32_t* out_parent;       // [B][K]
    int32_t* out_token;        // [B][K]
    float* out_score;          // [B][K]
    int32_t* out_status;       // [B] or null
    int B, W, V, K, nb, Lsh;   // chunks of 2^Lsh lanes
    int pad_token;
};

__device__ __forceinline__ uint32_t beam_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ bool beam_t_ok(float T) { return T == 0.f || (T >= SV_TEMPERATURE_MIN && T <= FLT_MAX); }

// Integer offset of a batch's sum: of its maximum, kept finite where a batch holds only
// the type's lowest values (its sum is then 0).  T = 0 (khi = 1) needs the NaN test only.
// Up to kBeamOffset the offset is within 48 of the maximum's exponent (fp32 steps by up to
// 32 there, and klo adds up to 32), so a batch's sum lies in fp32's range and keeps terms
// down to 2^-78 of the largest.  Beyond it the sum may be anything, 0 or infinite
// included: such a batch counts for nothing beside a maximum within the bound, and
// where the row's own maximum is beyond it the normaliser is taken again in fp64.
constexpr float kBeamOffset = 0x1p28f;
__device__ __forceinline__ float beam_offset(float m, float khi)
{
    return m == -INFINITY ? 0.f : fmaxf(ceilf(__fmul_rn(m, khi)), -3e38f);
}

__device__ __forceinline__ void beam_k(float T, float* khi, float* klo)
{
    *khi = 1.f;
    *klo = 0x1p-60f;
    if (T > 0.f) split_k(T, khi, klo);
}

// max over the warp (NaN ignored unless all are)
__device__ __forceinline__ float beam_warp_max(float x)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

// Row elements [i, i + VEC), element by element; -inf past V.
template <int ESZ>
__device__ __noinline__ uint4 beam_ld_edge(const unsigned char* p, int i, int V)
{
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

// Row elements [i, i + VEC), -inf past V, of a row that may start off a 16-byte
// boundary: only blocks that hold an element of the row are read, and no byte past `end`.
template <int ESZ, bool AL>
__device__ __forceinline__ uint4 beam_ld(const unsigned char* row, int i, int V, const unsigned char* end)
{
    constexpr uint32_t ninf = ESZ == 2 ? 0xff80ff80u : 0xff800000u;
    if (i >= V) return make_uint4(ninf, ninf, ninf, ninf);
    const unsigned char* p = row + (size_t)i * ESZ;
    if (AL) return ld_stream(reinterpret_cast<const uint4*>(p));
    const unsigned sh = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u);
    const unsigned char* a = p - sh;
    if (i + 16 / ESZ <= V && a + 32 <= end)
        return shift16(__ldg(reinterpret_cast<const uint4*>(a)), __ldg(reinterpret_cast<const uint4*>(a) + 1), sh);
    return beam_ld_edge<ESZ>(p, i, V);
}

// Floats as integers of the same order (-0 first made +0).
__device__ __forceinline__ unsigned beam_ord(float v)
{
    const unsigned u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float beam_unord(unsigned o)
{
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

// (value, index) as one integer of the candidates' order: larger value, then smaller
// index; 0 for -inf and NaN, which are no candidates.
__device__ __forceinline__ unsigned long long beam_key(float v, int i)
{
    return v > -INFINITY ? (unsigned long long)beam_ord(v) << 32 | (0xffffffffu - (unsigned)i) : 0ull;
}

__device__ __forceinline__ unsigned long long beam_warp_max64(unsigned long long k)
{
    const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(k >> 32));
    const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(k >> 32) == hi ? (unsigned)k : 0u);
    return (unsigned long long)hi << 32 | lo;
}

// Bytes of shared memory a warp of sv_beam_rows needs: two batches, and the block that
// an unaligned row's last vector reaches into.
constexpr int kBeamSlot = kBeamNV * 32 + 1;
constexpr int kBeamWarpBytes = 2 * kBeamSlot * 16;

// AL: every row starts on a 16-byte boundary (its length is then whole vectors);
// otherwise a vector comes from the two 16-byte blocks it lies in.  Only blocks that
// hold an element of the row are read, and no byte past the logits' end.  The next
// batch's blocks are copied to the warp's shared memory while this one is worked on;
// nothing is shared between warps.
template <int ESZ, bool AL>
__global__ void __launch_bounds__(kBeamThreads, 3) sv_beam_rows(BeamArgs g, int spans)
{
    constexpr int VEC = 16 / ESZ, NV = kBeamNV, STEP = NV * 32 * VEC;  // tokens of a batch
    constexpr uint32_t ninf = ESZ == 2 ? 0xff80ff80u : 0xff800000u;
    extern __shared__ __align__(16) unsigned char beam_rows_dyn[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = g.B * g.W;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < g.B; i += gridDim.x * blockDim.x) g.ticket[i] = 0u;
    // this warp's span of the rows' batches
    const long long span = (long long)blockIdx.x * (blockDim.x >> 5) + warp, batches = (long long)rows * g.nb;
    if (span >= spans) return;
    const long long first = span * batches / spans;
    int left = (int)((span + 1) * batches / spans - first);
    int row = (int)(first / g.nb), batch = (int)(first % g.nb);
    const unsigned char* base = static_cast<const unsigned char*>(g.logits);
    const unsigned char* end = base + (size_t)rows * g.V * ESZ;
    const int L = 1 << g.Lsh, cpv = 32 >> g.Lsh;  // lanes of a chunk, chunks of a warp's vector
    uint4* const slots = reinterpret_cast<uint4*>(beam_rows_dyn) + warp * 2 * kBeamSlot;

    // a row's temperature, and whether any candidate comes from its logits
    auto look = [&](int r, float& T) {
        T = __ldg(g.temperature + r / g.W);
        const float sc = __ldg(g.score + r);
        return beam_t_ok(T) && sc > -INFINITY && sc < INFINITY && !(g.frozen && __ldg(g.frozen + r));
    };
    auto copy = [&](int r, int bt, int slot) {
        const unsigned char* rp = base + (size_t)r * g.V * ESZ;
        const unsigned sh = AL ? 0u : (unsigned)(reinterpret_cast<uintptr_t>(rp) & 15u);
        const unsigned char* p = rp - sh + (size_t)(bt * NV * 32 + lane) * 16;
        const uint32_t to = beam_smem(slots + slot * kBeamSlot + lane);
        if ((bt + 1) * STEP <= g.V && (AL || p - lane * 16 + (NV * 32 + 1) * 16 <= end)) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + j * 512), "l"(p + j * 512) : "memory");
            if (!AL && lane == 0)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + NV * 512), "l"(p + NV * 512) : "memory");
        } else {
            const unsigned char* stop = rp + (size_t)g.V * ESZ;  // past the row
#pragma unroll 1
            for (int j = 0; j <= NV; ++j) {
                if (j == NV && (AL || lane)) break;
                const unsigned char* q = p + j * 512;
                if (q < stop) {
                    const int bytes = (int)min((long long)16, (long long)(end - q));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + j * 512), "l"(q), "r"(bytes) : "memory");
                } else {
                    slots[slot * kBeamSlot + j * 32 + lane] = make_uint4(ninf, ninf, ninf, ninf);
                }
            }
        }
    };
    float T, Tn = 0.f, Tk = -1.f, khi = 1.f, klo = 0.f;
    int slot = 0;
    copy(row, batch, 0);  // before it is known whether the row counts
    asm volatile("cp.async.commit_group;" ::: "memory");
    bool live = look(row, T), liven = false;
    while (true) {
        // the next batch
        const bool turn = batch + 1 == g.nb;
        if (left > 1) {
            if (turn) {
                copy(row + 1, 0, slot ^ 1);
                liven = look(row + 1, Tn);
            } else if (live) {
                copy(row, batch + 1, slot ^ 1);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (live) {
            if (T != Tk) {
                beam_k(T, &khi, &klo);
                Tk = T;
            }
            const uint4* at = slots + slot * kBeamSlot + lane;
            uint4 v[NV];
            if (AL) {
#pragma unroll
                for (int j = 0; j < NV; ++j) v[j] = at[j * 32];
            } else {
                __syncwarp();  // the other lanes' copies
                const unsigned sh = (unsigned)(reinterpret_cast<uintptr_t>(base + (size_t)row * g.V * ESZ) & 15u);
#pragma unroll
                for (int j = 0; j < NV; ++j) v[j] = shift16(at[j * 32], at[j * 32 + 1], sh);
                if ((batch + 1) * STEP > g.V) {  // elements past the row
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int n = (g.V - (batch * STEP + (j * 32 + lane) * VEC)) * ESZ;  // bytes of it
                        uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (4 * k >= n) x[k] = ninf;
                            else if (ESZ == 2 && 4 * k + 2 >= n) x[k] = (x[k] & 0xffffu) | 0xff800000u;
                        }
                        v[j] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            float m[NV], mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) m[j] = vec_max<ESZ>(v[j]);
            float* cmax = g.cmax + ((size_t)row * g.nb + batch) * (NV * cpv);
            if (L == 32) {
                float mine = 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    m[j] = beam_warp_max(m[j]);
                    mx = fmaxf(mx, m[j]);
                    mine = lane == j ? m[j] : mine;
                }
                if (lane < NV) cmax[lane] = mine;
            } else {
                for (int o = 1; o < L; o <<= 1)
#pragma unroll
                    for (int j = 0; j < NV; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if ((lane & (L - 1)) == 0) cmax[j * cpv + (lane >> g.Lsh)] = m[j];
                    mx = fmaxf(mx, m[j]);
                }
                mx = beam_warp_max(mx);
            }
            unsigned long long acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = pack2(0.f, 0.f);
            lazy_exps_add<ESZ, NV>(acc, v, khi, klo, beam_offset(mx, khi));
            const float s = lazy_warp_sum(acc);
            if (lane == 0) g.part[(size_t)row * g.nb + batch] = make_float2(mx, s);
        }
        if (--left <= 0) return;
        slot ^= 1;
        if (turn) {
            batch = 0;
            ++row;
            live = liven;
            T = Tn;
        } else {
            ++batch;
        }
    }
}

// The want best of n keys (larger first), one after the other, by the whole CTA:
// each(f) calls f on every key of this thread; out(k, key) takes the k-th, 0 for none.
template <class Each, class Out>
__device__ __forceinline__ void pick_one_by_one(int want, unsigned long long* s_tmp, Each each, Out out)
{
    unsigned long long last = ~0ull;
    for (int k = 0; k < want; ++k) {
        unsigned long long best = 0ull;
        each([&](unsigned long long key) {
            if (key < last && key > best) best = key;
        });
        best = beam_warp_max64(best);
        if ((threadIdx.x & 31) == 0) s_tmp[threadIdx.x >> 5] = best;
        __syncthreads();
        best = s_tmp[0];
        for (int i = 1; i < kPickWarps; ++i) best = max(best, s_tmp[i]);
        __syncthreads();
        last = best;
        if (threadIdx.x == 0) out(k, best);
    }
}

// How many of s_key[0, n) rank before number `me`: larger, or equal and earlier.  n is
// taken up to a multiple of 4; s_key is 16-byte aligned and holds zeros from n on.
__device__ __forceinline__ int pick_rank(const unsigned long long* s_key, int n, unsigned long long key, int me)
{
    int rank = 0;
#pragma unroll 2
    for (int o = 0; o < n; o += 4) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s_key + o);
        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(s_key + o + 2);
        rank += a.x > key || (a.x == key && o < me);
        rank += a.y > key || (a.y == key && o + 1 < me);
        rank += c.x > key || (c.x == key && o + 2 < me);
        rank += c.y > key || (c.y == key && o + 3 < me);
    }
    return rank;
}

// log(sum exp((l - top) / T)) of a row by the whole CTA, in fp64 and in a fixed order: for
// rows whose logits / T are beyond what the pass's offsets hold.  NaN where the row has
// one, or top / T leaves fp32's range.  64 x 8 x 128256 bf16 with every row such a one: 133
// us a selection, against 39 with none.
template <int ESZ, bool AL>
__device__ __noinline__ double pick_lse_wide(const BeamArgs& g, int row, float top, float T, double* s_sum)
{
    constexpr int VEC = 16 / ESZ;
    const unsigned char* base = static_cast<const unsigned char*>(g.logits);
    const unsigned char* end = base + (size_t)g.B * g.W * g.V * ESZ;
    const double inv = 1.0 / (double)T;
    double S = fabs((double)top / (double)T) <= FLT_MAX ? 0.0 : NAN;
#pragma unroll 1
    for (int i = threadIdx.x * VEC; i < g.V; i += kPickThreads * VEC) {
        float x[VEC];
        unpack<ESZ>(beam_ld<ESZ, AL>(base + (size_t)row * g.V * ESZ, i, g.V, end), x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const double y = ((double)x[e] - (double)top) * inv;
            if (!(y < -746.0)) S += exp(y);  // below that exp is 0; NaN is taken
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    __syncthreads();  // s_sum's earlier values have been read
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = S;
    __syncthreads();
    S = s_sum[0];
    for (int i = 1; i < kPickWarps; ++i) S += s_sum[i];
    return log(S);
}

// A value into the first CTA of the cluster's copy of a shared variable.
__device__ __forceinline__ void pick_first(const void* p, double v)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.f64 [a], %1;\n\t}" ::"r"(beam_smem(p)), "d"(v)
                 : "memory");
}

__device__ __forceinline__ void pick_first(const void* p, int v)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t}" ::"r"(beam_smem(p)), "r"(v)
                 : "memory");
}

// CL: the rows of a sequence are one cluster (W <= 8) and hand their candidates to its
// first CTA's shared memory; otherwise through the workspace and a ticket (64 x 8 x 128256
// bf16, K = 8: 39.3 us in all by ticket, 37.5 by cluster).
template <int ESZ, bool AL, bool CL>
__global__ void __launch_bounds__(kPickThreads) sv_beam_pick(const __grid_constant__ BeamArgs g)
{
    constexpr int VEC = 16 / ESZ, NU = 4, GROUPS = 64;
    __shared__ float s_group[GROUPS];
    __shared__ double s_sum[kPickWarps], s_lse;
    __shared__ float s_top[kPickWarps];
    __shared__ __align__(16) unsigned long long s_cand[kBeamCap + 4];
    __shared__ __align__(16) unsigned long long s_best[kPickThreads];
    __shared__ unsigned long long s_tmp[kPickWarps];
    __shared__ int s_at[kPickThreads];
    __shared__ int s_sel[kPickChunks];
    __shared__ float s_tau, s_low;
    __shared__ int s_n, s_m, s_last;
    __shared__ double s_key[CL ? kPickCluster * SV_MAX_BEAMS : 1];  // CL, first CTA: [W][K]
    __shared__ int s_tok[CL ? kPickCluster * SV_MAX_BEAMS : 1];
    __shared__ int2 s_info[CL ? kPickCluster : 1];
    if (CL) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
    const int row = blockIdx.x, b = row / g.W, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nch = g.nb * kBeamNV << (5 - g.Lsh), CH = VEC << g.Lsh, L = 1 << g.Lsh;
    const float T = __ldg(g.temperature + b), sc = __ldg(g.score + row);
    const bool frozen = g.frozen && __ldg(g.frozen + row), t_ok = beam_t_ok(T);
    float khi, klo;
    beam_k(t_ok ? T : 0.f, &khi, &klo);
    // candidate k of this row, and how many there are
    auto keep = [&](int k, double key, int token) {
        if (CL) {
            const int c = (row - b * g.W) * g.K + k;
            pick_first(&s_key[c], key);
            pick_first(&s_tok[c], token);
        } else {
            g.key[(size_t)row * g.K + k] = key;
            g.tok[(size_t)row * g.K + k] = token;
        }
    };
    if (tid == 0) { s_n = 0; s_m = 0; }
    if (CL) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int cnt = 0, bad = 0;
    if (!(sc < INFINITY)) {
        bad = SV_ROW_BAD_SCORE;
    } else if (sc == -INFINITY) {
    } else if (frozen) {
        cnt = 1;
        if (tid == 0) keep(0, (double)sc, g.pad_token);
    } else if (t_ok) {
        // ---- the chunks' maxima and the row's normaliser: batch sums against the largest
        // offset, in fp64
        const float* cmax = g.cmax + (size_t)row * nch;
        const float2* part = g.part + (size_t)row * g.nb;
        float best = -INFINITY, m = -INFINITY;
#pragma unroll 8
        for (int c = tid; c < nch; c += kPickThreads) best = fmaxf(best, cmax[c]);
        const float2 p0 = tid < g.nb ? part[tid] : make_float2(-INFINITY, 0.f);
        const int want = T > 0.f ? g.K : 1;  // T = 0: all mass on the first argmax
        // 64 groups of two threads, 32 of four where they bound the few wanted well enough
        const int per = want <= 8 ? 4 : 2, groups = kPickThreads / per;
        m = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
        if (per == 4) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (tid % per == 0) s_group[tid / per] = m;
        m = beam_warp_max(m);
        if (lane == 0) s_top[warp] = m;
        __syncthreads();
        float top = s_top[0];
#pragma unroll
        for (int i = 1; i < kPickWarps; ++i) top = fmaxf(top, s_top[i]);
        const float MK = beam_offset(top, khi);
        {
            // the want-th largest of the groups' maxima bounds the want-th chunk's from
            // below; each warp places its own quarter of them
            const float x0 = s_group[lane], x1 = groups > 32 ? s_group[32 + lane] : -INFINITY;
            const int first = warp * (groups / kPickWarps);
            const float mine = first < 32 ? x0 : x1;
#pragma unroll 4
            for (int q = 0; q < groups / kPickWarps; ++q) {
                const int me = first + q;
                const float y = __shfl_sync(0xffffffffu, mine, me & 31);
                const unsigned b0 = __ballot_sync(0xffffffffu, x0 > y || (x0 == y && lane < me));
                const unsigned b1 = __ballot_sync(0xffffffffu, x1 > y || (x1 == y && 32 + lane < me));
                if (__popc(b0) + __popc(b1) == want - 1 && lane == 0) s_tau = y;
            }
        }
        double S = 0.0;
        {
            // (a batch without weight may hold an infinite sum; NaN stays)
            auto add = [&](const float2& p) {
                const double weight = p.x == -INFINITY ? 1.0 : pow2d(beam_offset(p.x, khi) - MK);
                if (weight > 0.0 || p.y != p.y) S += (double)p.y * weight;
            };
            add(p0);
            for (int t = tid + kPickThreads; t < g.nb; t += kPickThreads) add(part[t]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
            if (lane == 0) s_sum[warp] = S;
        }
        __syncthreads();
        S = s_sum[0];
#pragma unroll
        for (int i = 1; i < kPickWarps; ++i) S += s_sum[i];
        // (a NaN makes S NaN; an all -inf batch has sum 0)
        const bool finite = top > -INFINITY && top < INFINITY;
        const bool wide = T > 0.f && finite && !(fabsf(MK) <= kBeamOffset);
        if (wide) S = pick_lse_wide<ESZ, AL>(g, row, top, T, s_sum);
        if (!finite || S != S) {
            bad = SV_ROW_BAD_LOGITS;
        } else {
            // ---- the chunks that hold the `want` best logits: those at or above the bound, a
            // few more than `want`; where ties make them many, exactly the `want` best
            // (and, meanwhile, the normaliser's logarithm, of logits taken from `ref`)
            const float tau = s_tau;
            const double ref = wide ? (double)top : 0.0;
            if (tid == kPickThreads - 1) s_lse = wide ? S : ((double)MK + log2(S)) * kLn2;
            if (best >= tau) {
                for (int c = tid; c < nch; c += kPickThreads) {
                    const float x = cmax[c];
                    if (x >= tau && x > -INFINITY) {
                        const int at = atomicAdd(&s_n, 1);
                        if (at < kPickChunks) s_sel[at] = c;
                    }
                }
            }
            __syncthreads();
            int n = s_n;
            float low = tau;  // every logit wanted is at or above it
            if (n > kPickChunks) {
                n = want;
                pick_one_by_one(want, s_tmp,
                                [&](auto f) {
                                    for (int c = tid; c < nch; c += kPickThreads) f(beam_key(cmax[c], c));
                                },
                                [&](int k, unsigned long long k1) {
                                    s_sel[k] = (int)(0xffffffffu - (unsigned)k1);
                                    s_low = beam_unord((unsigned)(k1 >> 32));
                                });
                __syncthreads();
                low = s_low;
            }
            // ---- the logits of the chosen chunks
            const unsigned char* base = static_cast<const unsigned char*>(g.logits);
            const unsigned char* end = base + (size_t)g.B * g.W * g.V * ESZ;
            const unsigned char* rp = base + (size_t)row * g.V * ESZ;
            const int vectors = n << g.Lsh;
            // first token of vector t of the chosen
            auto index = [&](int t) { return t < vectors ? s_sel[t >> g.Lsh] * CH + (t & (L - 1)) * VEC : g.V; };
            for (int t0 = tid; t0 < vectors; t0 += kPickThreads * NU) {
                uint4 v[NU];
#pragma unroll
                for (int u = 0; u < NU; ++u) v[u] = beam_ld<ESZ, AL>(rp, index(t0 + u * kPickThreads), g.V, end);
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    float x[VEC];
                    unpack<ESZ>(v[u], x);
                    unsigned hit = 0;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) hit |= (x[e] >= low && x[e] > -INFINITY ? 1u : 0u) << e;
                    if (hit) {
                        const int i = index(t0 + u * kPickThreads);
                        int at = atomicAdd(&s_m, __popc(hit));
                        do {
                            const int e = __ffs(hit) - 1, word = e * ESZ / 4;
                            hit &= hit - 1;
                            uint32_t q = word == 0 ? v[u].x : (word == 1 ? v[u].y : (word == 2 ? v[u].z : v[u].w));
                            if (ESZ == 2) q = (e & 1) ? q & 0xffff0000u : q << 16;
                            if (at < kBeamCap) s_cand[at] = beam_key(__uint_as_float(q), i + e);
                            ++at;
                        } while (hit);
                    }
                }
            }
            __syncthreads();
            n = s_m;
            cnt = min(n, want);
            const double lse = s_lse;
            auto put = [&](int k, unsigned long long k1) {
                const double l = (double)beam_unord((unsigned)(k1 >> 32));
                keep(k, T > 0.f ? (double)sc + ((l - ref) / (double)T - lse) : (double)sc, (int)(0xffffffffu - (unsigned)k1));
            };
            if (n <= kBeamCap) {
                if (tid < 4) s_cand[n + tid] = 0ull;
                __syncthreads();
                for (int c = tid; c < n; c += kPickThreads) {
                    const unsigned long long k1 = s_cand[c];
                    const int rank = pick_rank(s_cand, n, k1, c);
                    if (rank < want) put(rank, k1);
                }
            } else {  // many equal logits
                pick_one_by_one(want, s_tmp,
                                [&](auto f) {
                                    for (int t = tid; t < vectors; t += kPickThreads) {
                                        const int i = index(t);
                                        float x[VEC];
                                        unpack<ESZ>(beam_ld<ESZ, AL>(rp, i, g.V, end), x);
#pragma unroll
                                        for (int e = 0; e < VEC; ++e) f(beam_key(x[e], i + e));
                                    }
                                },
                                put);
            }
        }
    }
    // ---- the sequence's first CTA, or the last one to finish, joins the rows
    if (CL) {
        if (tid == 0) {
            pick_first(&s_info[row - b * g.W].x, cnt);
            pick_first(&s_info[row - b * g.W].y, bad);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (row != b * g.W) return;
    } else if (g.W > 1) {
        if (tid == 0) g.row_info[row] = make_int2(cnt, bad);
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(g.ticket + b, 1u) == (unsigned)g.W - 1u;
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    } else {
        if (tid == 0) g.row_info[row] = make_int2(cnt, bad);
        __syncthreads();  // this row is the sequence
    }
    const size_t row0 = (size_t)b * g.W;
    // the keys, as integers of their order (0: none), where the candidates' memory is no
    // longer needed; candidate c = w K + k, so ties go to the smaller c
    const int all = g.W * g.K;
    int* s_cnt = s_sel;
    const int2 info = tid < g.W ? (CL ? s_info[CL ? tid : 0] : __ldcg(g.row_info + row0 + tid)) : make_int2(0, 0);
    if (tid < g.W) s_cnt[tid] = info.x;
    if (warp == 0) {
        const unsigned st = __reduce_or_sync(0xffffffffu, (unsigned)info.y);
        if (g.out_status && lane == 0) g.out_status[b] = (int)(st | (t_ok ? 0u : SV_ROW_BAD_TEMPERATURE));
    }
    if (tid < 4) s_cand[all + tid] = 0ull;
    __syncthreads();
    unsigned long long best = 0ull;
    for (int c = tid; c < all; c += kPickThreads) {
        const int w = c / g.K;
        unsigned long long o = 0ull;
        if (c - w * g.K < s_cnt[w]) {
            const unsigned long long u = (unsigned long long)__double_as_longlong((CL ? s_key[CL ? c : 0] : __ldcg(g.key + row0 * g.K + c)) + 0.0);
            o = u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
        }
        s_cand[c] = o;
        best = max(best, o);
    }
    auto put = [&](int c, unsigned long long mine, int place) {
        if (place >= g.K) return;
        const size_t at = (size_t)b * g.K + place;
        g.out_parent[at] = c / g.K;
        g.out_token[at] = CL ? s_tok[CL ? c : 0] : __ldcg(g.tok + row0 * g.K + c);
        g.out_score[at] = (float)__longlong_as_double((long long)(mine ^ ((mine >> 63) ? 0x8000000000000000ull : ~0ull)));
    };
    bool rank_all = all <= kPickThreads;
    if (!rank_all) {
        // many candidates: only those at or above the K-th of the threads' largest matter
        s_best[tid] = best;
        if (tid == 0) s_n = 0;
        __syncthreads();
        if (pick_rank(s_best, kPickThreads, best, tid) == g.K - 1) s_tmp[0] = best;
        __syncthreads();
        const unsigned long long floor = max(1ull, s_tmp[0]);
        for (int c = tid; c < all; c += kPickThreads)
            if (s_cand[c] >= floor) {
                const int at = atomicAdd(&s_n, 1);
                if (at < kPickThreads) {
                    s_best[at] = s_cand[c];
                    s_at[at] = c;
                }
            }
        __syncthreads();
        const int n = s_n;
        rank_all = n > kPickThreads;  // (many equal keys)
        if (tid < n && !rank_all) {
            const unsigned long long mine = s_best[tid];
            const int c = s_at[tid];
            int place = 0;
#pragma unroll 4
            for (int o = 0; o < n; ++o) place += s_best[o] > mine || (s_best[o] == mine && s_at[o] < c);
            put(c, mine, place);
        }
    }
    __syncthreads();
    if (rank_all)
        for (int c = tid; c < all; c += kPickThreads)
            if (s_cand[c]) put(c, s_cand[c], pick_rank(s_cand, all, s_cand[c], c));
    int total = 0;
    for (int w = 0; w < g.W; ++w) total += s_cnt[w];
    if (tid >= total && tid < g.K) {
        const size_t at = (size_t)b * g.K + tid;
        g.out_parent[at] = -1;
        g.out_token[at] = -1;
        g.out_score[at] = -INFINITY;
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
