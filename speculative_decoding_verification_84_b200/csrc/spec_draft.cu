// spec_draft.cu -- C ABI of the draft's step upstream of verification: the 8-bit
// head (sv_q8.cuh), and the selection of a tree's next level with the reordering of
// the draft's states (sv_beam.cuh).  The operations are specified in
// include/spec_verify.h.
#include "spec_verify.h"

#include <cuda.h>  // CUtensorMap: driver calls go through entry points
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "sv_common.cuh"
#include "sv_host.cuh"
#include "sv_q8.cuh"
#include "sv_beam.cuh"

namespace {

using namespace sv;

inline bool dt_ok(sv_dtype dt) { return dt == SV_DTYPE_F32 || dt == SV_DTYPE_BF16; }

// Lets a kernel have `bytes` of dynamic shared memory, once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<bool> (&ready)[kMaxDevices])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    if (known && ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && known) ready[dev].store(true, std::memory_order_release);
    return e;
}

// ----------------------------------------------------------------------------- rows to int8

constexpr int kQ8RowsSmemMax = 208 * 1024;

size_t q8_rows_smem(int nv, int threads, int rows, bool res, bool al)
{
    return (size_t)16 * q8_rows_kept(res, al) * rows * q8_row_blocks(nv, threads);
}

template <int ESZ, int NV, int MAXT, bool RES, bool AL>
cudaError_t q8_rows_go(const Q8RowsArgs& g, int threads, cudaStream_t st)
{
    // rows of one warp: eight to a CTA
    const dim3 block(threads, threads == 32 ? 8 : 1);
    const int all = threads * (int)block.y;
    const size_t smem = q8_rows_smem(NV, threads, (int)block.y, RES, AL);
    if (smem > 40 * 1024) {  // more than a kernel has without asking, static part included
        static std::atomic<bool> ready[kMaxDevices];
        const cudaError_t e = allow_smem(sv_q8_rows<ESZ, NV, MAXT, RES, AL>, kQ8RowsSmemMax, ready);
        if (e != cudaSuccess) return e;
    }
    // as many CTAs as are resident at once, each walking rows
    static std::atomic<int> regs;
    int nreg = regs.load(std::memory_order_relaxed);
    if (!nreg) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, sv_q8_rows<ESZ, NV, MAXT, RES, AL>);
        if (e != cudaSuccess) return e;
        nreg = (a.numRegs + 7) / 8 * 8;
        regs.store(nreg, std::memory_order_relaxed);
    }
    const long long fit = std::min<long long>(std::min(2048 / all, 65536 / (nreg * all)), (long long)(226 * 1024 / (smem + 2048)));
    const long long grid = std::min<long long>(cdiv(g.M, block.y), device_sm_count() * std::max<long long>(1, fit));
    sv_q8_rows<ESZ, NV, MAXT, RES, AL><<<(unsigned)grid, block, smem, st>>>(g);
    return cudaGetLastError();
}

// A row by one warp, without barriers across warps, where 4 vectors a thread are enough,
// else by up to 256 threads with as few vectors each as that allows, else by up to 1024;
// rows that shared memory cannot hold three of, from memory, twice.
template <int ESZ, bool RES, bool AL>
cudaError_t q8_rows_launch(const Q8RowsArgs& g, cudaStream_t st)
{
    const long long pieces = cdiv((long long)g.d * ESZ, 16);
    const int room = pieces <= 32 * 4 ? 32 : 256;
    const int nv = pieces <= room ? 1 : (pieces <= 2 * room ? 2 : 4);
    const long long threads = cdiv(cdiv(pieces, nv), 32) * 32;
    if (threads > 1024 || q8_rows_smem(nv, (int)threads, threads == 32 ? 8 : 1, RES, AL) > (size_t)kQ8RowsSmemMax) {
        sv_q8_rows_long<ESZ><<<(unsigned)g.M, 1024, 0, st>>>(g);
        return cudaGetLastError();
    }
    if (threads > 256) return q8_rows_go<ESZ, 4, 1024, RES, AL>(g, (int)threads, st);
    if (nv == 1) return q8_rows_go<ESZ, 1, 256, RES, AL>(g, (int)threads, st);
    if (nv == 2) return q8_rows_go<ESZ, 2, 256, RES, AL>(g, (int)threads, st);
    return q8_rows_go<ESZ, 4, 256, RES, AL>(g, (int)threads, st);
}

template <int ESZ>
cudaError_t q8_rows_dt(const Q8RowsArgs& g, cudaStream_t st)
{
    const bool al = (long long)g.d * ESZ % 16 == 0;  // every row on a 16-byte boundary
    if (g.r) return al ? q8_rows_launch<ESZ, true, true>(g, st) : q8_rows_launch<ESZ, true, false>(g, st);
    return al ? q8_rows_launch<ESZ, false, true>(g, st) : q8_rows_launch<ESZ, false, false>(g, st);
}

sv_status q8_rows(const Q8RowsArgs& g, sv_dtype dt, cudaStream_t st)
{
    const cudaError_t e = dt == SV_DTYPE_BF16 ? q8_rows_dt<2>(g, st) : q8_rows_dt<4>(g, st);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status q8_rows_check(const void* x, sv_dtype dt, int M, int d, const void* q, int ldq, const void* scale)
{
    if (!x || !q || !scale || M < 1 || M > SV_Q8_MAX_M || d < 1 || d > SV_Q8_MAX_K || ldq < d || ldq % 16) return SV_ERR_INVALID_ARG;
    if (!dt_ok(dt)) return SV_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return SV_ERR_MISALIGNED;
    return SV_OK;
}

// ----------------------------------------------------------------------------- the product

// Tensor map of a row-major int8 [rows][K] matrix of row pitch ld, in boxes of
// kQ8BK bytes x box_rows, 128-byte swizzle; elements past K and rows read as zero.
bool q8_map(CUtensorMap* m, const void* base, long long rows, long long K, long long ld, int box_rows)
{
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)kQ8BK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of SMs resident at once on the current device (an SM without a partner in its
// GPC has none); 0 and *e on a CUDA error.
template <int ESZ>
int q8_resident_pairs(cudaError_t* e)
{
    static std::atomic<int> resident[kMaxDevices];
    static std::atomic<bool> ready[kMaxDevices];
    if ((*e = allow_smem(sv_q8_gemm<ESZ, true>, kQ8SmemMax, ready)) != cudaSuccess) return 0;
    int dev = 0;
    if ((*e = cudaGetDevice(&dev)) != cudaSuccess) return 0;
    const bool known = dev >= 0 && dev < kMaxDevices;
    int n = known ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (device_sm_count() / 2)));
    cfg.blockDim = dim3(kQ8Threads);
    cfg.dynamicSmemBytes = kQ8SmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    *e = cudaOccupancyMaxActiveClusters(&n, sv_q8_gemm<ESZ, true>, &cfg);
    if (*e == cudaSuccess && n < 1) *e = cudaErrorInvalidConfiguration;
    if (*e != cudaSuccess) return 0;
    if (known) resident[dev].store(n, std::memory_order_relaxed);
    return n;
}

// How the product is cut.
//  * Pairs of SMs where an SM has 32 K blocks or more to walk; the pair's extra steps at
//    start and end cost about 1.3 us (37 x 1001 x 3001: 6.5 us on single SMs, 8.0 on
//    pairs; 1 x 4096 x 32000: 24.5 and 23.9; 2048 x 4096 x 64000: 441 and 384).
//  * As few accumulators of 256 tokens as hold the batch, all of one size; more and
//    smaller ones where the tiles would leave SMs idle.
//  * Two accumulators to a tile where they are the whole batch, so that the weights are
//    read once, if a third fits beside them (the next tile then starts while these are
//    stored: at most 160 tokens each) and the rounds of tiles are not made worse by it: a
//    tile of two takes 1.8 times as long (320 x 4096: V = 128256 7 rounds 140 us against
//    14 of 156; V = 64000 4 of 82 against 7 of 81).
//  * Two K blocks to a stage where four such stages fit, which halves the waits and
//    commits; else one (2048 x 4096 x 64000: 384 us with one, 398 with two; 1 x 4096 x
//    64000: 46.0 and 44.3).
void q8_cut(Q8GemmArgs& g, int sms, int resident, bool* pairs)
{
    const int kbs = (int)cdiv(g.K, kQ8BK);
    const long long accs = cdiv(g.M, kQ8MaxNT);
    *pairs = cdiv(accs * cdiv(g.V, 2 * kQ8BM), resident) * kbs >= 32;
    const int unit = *pairs ? 32 : 16;
    const long long units = *pairs ? resident : sms;  // tiles at a time
    g.v_tiles = (int)cdiv(g.V, *pairs ? 2 * kQ8BM : kQ8BM);
    long long parts = accs;
    if (parts * g.v_tiles < units) parts = std::min<long long>(units / g.v_tiles, std::max<long long>(accs, cdiv(g.M, 32)));
    g.nt = (int)(cdiv(cdiv(g.M, parts), unit) * unit);
    parts = cdiv(g.M, g.nt);
    g.groups = 1;
    if (*pairs && parts == 2 && g.nt <= 160 && 9 * cdiv(g.v_tiles, units) < 5 * cdiv(2LL * g.v_tiles, units)) g.groups = 2;
    g.m_tiles = (int)cdiv(parts, g.groups);
    g.buf_cols = (int)(cdiv(g.nt, 32) * 32);
    g.bufs = std::min(kQ8MaxBufs, 512 / g.buf_cols);
    g.tmem_cols = 32;
    while (g.tmem_cols < g.bufs * g.buf_cols) g.tmem_cols *= 2;
    const int block = kQ8WBytes + g.groups * (*pairs ? g.nt / 2 : g.nt) * kQ8BK;
    g.sub = 4 * kQ8MaxSub * block <= kQ8SmemMax - 1024 ? kQ8MaxSub : 1;
    g.stages = std::min(kQ8MaxStages, (kQ8SmemMax - 1024) / (g.sub * block));
}

template <int ESZ>
cudaError_t q8_gemm_launch(const void* a, long long lda, const void* w, long long ldw, Q8GemmArgs g, cudaStream_t st)
{
    cudaError_t e;
    const int sms = device_sm_count(), resident = q8_resident_pairs<ESZ>(&e);
    if (e != cudaSuccess) return e;
    bool pairs;
    q8_cut(g, sms, resident, &pairs);
    const int mine = pairs ? g.nt / 2 : g.nt;  // tokens of an accumulator in one CTA
    CUtensorMap tw, ta;
    if (!q8_map(&tw, w, g.V, g.K, ldw, kQ8BM) || !q8_map(&ta, a, g.M, g.K, lda, mine)) return cudaErrorInvalidValue;
    const long long tiles = (long long)g.m_tiles * g.v_tiles;
    const size_t smem = 1024 + (size_t)g.stages * g.sub * (kQ8WBytes + g.groups * mine * kQ8BK);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs ? 2 * std::min<long long>(tiles, resident) : std::min<long long>(tiles, sms)));
    cfg.blockDim = dim3(kQ8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (pairs) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = 2;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (g.overlap) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (pairs) return cudaLaunchKernelEx(&cfg, sv_q8_gemm<ESZ, true>, tw, ta, g);
    static std::atomic<bool> ready[kMaxDevices];
    if ((e = allow_smem(sv_q8_gemm<ESZ, false>, kQ8SmemMax, ready)) != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, sv_q8_gemm<ESZ, false>, tw, ta, g);
}

// after_norm: the launch before this one on the stream is the norm of `a`, which the
// product may overlap (its weights are older than that).
sv_status q8_gemm(const int8_t* a, int lda, const float* a_scale, const int8_t* w, int ldw, const float* w_scale, int M, int K,
                  int V, void* out, sv_dtype dt, int32_t* err, bool after_norm, cudaStream_t st)
{
    Q8GemmArgs g = {};
    g.out = out;
    g.a_scale = a_scale;
    g.w_scale = w_scale;
    g.err = err;
    g.M = M;
    g.V = V;
    g.K = K;
    g.overlap = after_norm ? 1 : 0;
    const cudaError_t e = dt == SV_DTYPE_BF16 ? q8_gemm_launch<2>(a, lda, w, ldw, g, st)
                                              : q8_gemm_launch<4>(a, lda, w, ldw, g, st);
    return e == cudaSuccess ? SV_OK : (e == cudaErrorInvalidValue ? SV_ERR_INVALID_ARG : SV_ERR_CUDA);
}

sv_status q8_gemm_check(const void* a, int lda, const void* a_scale, const void* w, int ldw, const void* w_scale, int M,
                        int K, int V, const void* out, sv_dtype dt, const void* err)
{
    if (!a || !a_scale || !w || !w_scale || !out || M < 1 || K < 1 || K > SV_Q8_MAX_K || V < 1 || V > SV_MAX_V ||
        lda < K || lda % 16 || ldw < K || ldw % 16 || M > SV_Q8_MAX_M ||
        cdiv(M, kQ8MaxNT) * cdiv(V, kQ8BM) > (1LL << 30))  // the tiles are counted in 32 bits
        return SV_ERR_INVALID_ARG;
    if (!dt_ok(dt)) return SV_ERR_UNSUPPORTED_DTYPE;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(err, 4))
        return SV_ERR_MISALIGNED;
    return SV_OK;
}

// ----------------------------------------------------------------------------- beams

struct BeamPlan {
    int nb, Lsh;
    size_t off_cmax, off_key, off_tok, off_info, off_ticket, total;
};

// Batches of a row, and the lanes of a chunk: the most for which a row still has 2 K
// chunks (the K best then hold little more than K logits at or above the least of
// their maxima); a single lane's vector where no width gives that (V below 16 K).
bool beam_plan(int B, int W, int V, int K, sv_dtype dt, BeamPlan* p)
{
    if (B < 1 || W < 1 || W > SV_MAX_BEAMS || K < 1 || K > SV_MAX_BEAMS || V < 1 || V > SV_BEAM_MAX_V || !dt_ok(dt))
        return false;
    const int vec = dt == SV_DTYPE_BF16 ? 8 : 4;
    p->nb = (int)cdiv(V, 32 * kBeamNV * vec);
    p->Lsh = 5;
    while (p->Lsh > 0 && cdiv(V, vec << p->Lsh) < 2 * K) --p->Lsh;
    const long long rows = (long long)B * W;
    if (rows > 0x7fffffffLL) return false;
    p->off_cmax = align256(sizeof(float2) * (size_t)rows * p->nb);
    p->off_key = p->off_cmax + align256(sizeof(float) * (size_t)rows * (size_t)(p->nb * kBeamNV << (5 - p->Lsh)));
    p->off_tok = p->off_key + align256(sizeof(double) * (size_t)rows * K);
    p->off_info = p->off_tok + align256(sizeof(int32_t) * (size_t)rows * K);
    p->off_ticket = p->off_info + align256(sizeof(int2) * (size_t)rows);
    p->total = p->off_ticket + align256(sizeof(unsigned) * (size_t)B);
    return true;
}

template <int ESZ, bool AL>
cudaError_t beam_go(const BeamArgs& g, cudaStream_t st)
{
    // one span of batches per resident warp (three CTAs of eight warps an SM), in smaller
    // CTAs where the batches are few, to reach every SM
    const long long batches = (long long)g.B * g.W * g.nb, sms = device_sm_count();
    const long long spans = std::min<long long>(batches, sms * 3 * (kBeamThreads / 32)), warps = std::min<long long>(kBeamThreads / 32, cdiv(spans, sms));
    static std::atomic<bool> ready[kMaxDevices];
    cudaError_t e = allow_smem(sv_beam_rows<ESZ, AL>, kBeamWarpBytes * (kBeamThreads / 32), ready);
    if (e != cudaSuccess) return e;
    sv_beam_rows<ESZ, AL><<<(unsigned)cdiv(spans, warps), (unsigned)(32 * warps), (size_t)(kBeamWarpBytes * warps), st>>>(g, (int)spans);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.B * g.W));
    cfg.blockDim = dim3(kPickThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.W;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (g.W == 1 || g.W > kPickCluster) return cudaLaunchKernelEx(&cfg, sv_beam_pick<ESZ, AL, false>, g);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sv_beam_pick<ESZ, AL, true>, g);
}

template <class VT>
cudaError_t reorder(ReorderArgs g, cudaStream_t st)
{
    const long long vecs = g.S * g.tb / (long long)sizeof(VT);
    g.tx = 8;
    while (g.tx < kReorderThreads && (long long)g.tx * kReorderU < vecs) g.tx *= 2;
    const long long tiles = cdiv(vecs, (long long)g.tx * kReorderU), groups = cdiv(g.chunks, kReorderThreads / g.tx);
    if (tiles > 0x7fffffffLL || groups > 0x7fffffffLL || tiles * groups > 0x7fffffffLL) return cudaErrorInvalidValue;
    sv_beam_reorder<VT><<<(unsigned)(tiles * groups), kReorderThreads, 0, st>>>(g);
    return cudaGetLastError();
}

}  // namespace

// ============================================================================= C ABI

extern "C" sv_status spec_verify_q8_quantize(const void* x, sv_dtype dt, int M, int K, int8_t* out_q, int ldq,
                                             float* out_scale, struct CUstream_st* stream)
{
    const sv_status s = q8_rows_check(x, dt, M, K, out_q, ldq, out_scale);
    if (s != SV_OK) return s;
    Q8RowsArgs g = {x, nullptr, nullptr, out_q, out_scale, nullptr, nullptr, ldq, M, K, 0.f, 0};
    return q8_rows(g, dt, (cudaStream_t)stream);
}

extern "C" sv_status spec_verify_q8_norm(const void* x, const void* residual, const void* weight, sv_dtype dt, float eps,
                                         int M, int d, int8_t* out_q, int ldq, float* out_scale, void* out_sum,
                                         void* out_normed, struct CUstream_st* stream)
{
    const sv_status s = q8_rows_check(x, dt, M, d, out_q, ldq, out_scale);
    if (s != SV_OK) return s;
    if (!(eps >= 0.f && eps <= FLT_MAX)) return SV_ERR_INVALID_ARG;
    if (!aligned(residual, 16) || !aligned(weight, 16) || !aligned(out_sum, 16) || !aligned(out_normed, 16))
        return SV_ERR_MISALIGNED;
    Q8RowsArgs g = {x, residual, weight, out_q, out_scale, out_sum, out_normed, ldq, M, d, eps, 1};
    return q8_rows(g, dt, (cudaStream_t)stream);
}

extern "C" sv_status spec_verify_q8_matmul(const int8_t* a, int lda, const float* a_scale, const int8_t* w, int ldw,
                                           const float* w_scale, int M, int K, int V, void* out, sv_dtype dt,
                                           int32_t* out_error, struct CUstream_st* stream)
{
    const sv_status s = q8_gemm_check(a, lda, a_scale, w, ldw, w_scale, M, K, V, out, dt, out_error);
    if (s != SV_OK) return s;
    return q8_gemm(a, lda, a_scale, w, ldw, w_scale, M, K, V, out, dt, out_error, false, (cudaStream_t)stream);
}

extern "C" size_t spec_verify_q8_head_workspace_size(int M, int d)
{
    if (M < 1 || M > SV_Q8_MAX_M || d < 1 || d > SV_Q8_MAX_K) return 0;
    return align256((size_t)M * (size_t)((d + 15) / 16 * 16)) + align256((size_t)M * sizeof(float));
}

extern "C" sv_status spec_verify_q8_head(const void* x, const void* residual, const void* weight, sv_dtype dt, float eps,
                                         const int8_t* w, int ldw, const float* w_scale, int M, int d, int V, void* out_sum,
                                         void* out_logits, sv_dtype out_dt, void* workspace, size_t workspace_bytes,
                                         int32_t* out_error, struct CUstream_st* stream)
{
    if (!workspace) return SV_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return SV_ERR_MISALIGNED;
    const size_t need = spec_verify_q8_head_workspace_size(M, d);
    if (!need) return SV_ERR_INVALID_ARG;
    if (workspace_bytes < need) return SV_ERR_WORKSPACE_TOO_SMALL;
    const int ld = (d + 15) / 16 * 16;
    int8_t* q = static_cast<int8_t*>(workspace);
    float* scale = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + align256((size_t)M * ld));
    // both halves' arguments, before anything is launched
    sv_status s = q8_gemm_check(q, ld, scale, w, ldw, w_scale, M, d, V, out_logits, out_dt, out_error);
    if (s != SV_OK) return s;
    s = spec_verify_q8_norm(x, residual, weight, dt, eps, M, d, q, ld, scale, out_sum, nullptr, stream);
    if (s != SV_OK) return s;
    return q8_gemm(q, ld, scale, w, ldw, w_scale, M, d, V, out_logits, out_dt, out_error, true, (cudaStream_t)stream);
}

extern "C" size_t spec_verify_beam_workspace_size(int B, int W, int V, int K, sv_dtype dt)
{
    BeamPlan p;
    return beam_plan(B, W, V, K, dt, &p) ? p.total : 0;
}

extern "C" sv_status spec_verify_beam_select(const void* logits, sv_dtype dt, const float* score, const float* temperature,
                                             const int32_t* frozen, int pad_token, int B, int W, int V, int K,
                                             int32_t* out_parent, int32_t* out_token, float* out_score,
                                             int32_t* out_row_status, void* workspace, size_t workspace_bytes,
                                             struct CUstream_st* stream)
{
    if (!logits || !score || !temperature || !out_parent || !out_token || !out_score || !workspace)
        return SV_ERR_INVALID_ARG;
    if (!dt_ok(dt)) return SV_ERR_UNSUPPORTED_DTYPE;
    BeamPlan p;
    if (!beam_plan(B, W, V, K, dt, &p)) return SV_ERR_INVALID_ARG;
    if (frozen && (pad_token < 0 || pad_token >= V)) return SV_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(score, 4) || !aligned(temperature, 4) || !aligned(frozen, 4) ||
        !aligned(out_parent, 4) || !aligned(out_token, 4) || !aligned(out_score, 4) || !aligned(out_row_status, 4) ||
        !aligned(workspace, 256))
        return SV_ERR_MISALIGNED;
    if (workspace_bytes < p.total) return SV_ERR_WORKSPACE_TOO_SMALL;
    BeamArgs g = {};
    g.logits = logits;
    g.score = score;
    g.temperature = temperature;
    g.frozen = frozen;
    g.part = static_cast<float2*>(workspace);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    g.cmax = reinterpret_cast<float*>(ws + p.off_cmax);
    g.key = reinterpret_cast<double*>(ws + p.off_key);
    g.tok = reinterpret_cast<int32_t*>(ws + p.off_tok);
    g.row_info = reinterpret_cast<int2*>(ws + p.off_info);
    g.ticket = reinterpret_cast<unsigned*>(ws + p.off_ticket);
    g.out_parent = out_parent;
    g.out_token = out_token;
    g.out_score = out_score;
    g.out_status = out_row_status;
    g.B = B;
    g.W = W;
    g.V = V;
    g.K = K;
    g.nb = p.nb;
    g.Lsh = p.Lsh;
    g.pad_token = pad_token;
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf = dt == SV_DTYPE_BF16, al = (long long)V * (bf ? 2 : 4) % 16 == 0;  // every row on a 16-byte boundary
    const cudaError_t e = bf ? (al ? beam_go<2, true>(g, st) : beam_go<2, false>(g, st))
                             : (al ? beam_go<4, true>(g, st) : beam_go<4, false>(g, st));
    return e == cudaSuccess ? SV_OK : (e == cudaErrorInvalidValue ? SV_ERR_INVALID_ARG : SV_ERR_CUDA);
}

extern "C" sv_status spec_verify_beam_reorder(const void* src, void* dst, const int32_t* parent, const int32_t* lengths,
                                              int L, int B, int W, int K, int H, long long S, long long token_bytes,
                                              struct CUstream_st* stream)
{
    if (!src || !dst || !parent || L < 1 || B < 1 || W < 1 || W > SV_MAX_BEAMS || K < 1 || K > SV_MAX_BEAMS || H < 1 ||
        S < 1 || token_bytes < 1)
        return SV_ERR_INVALID_ARG;
    long long chunks, block, in, out;
    if (__builtin_mul_overflow((long long)L * B, (long long)H, &chunks) || __builtin_mul_overflow(S, token_bytes, &block) ||
        __builtin_mul_overflow(chunks, block, &in) || __builtin_mul_overflow(in, (long long)K, &out) ||
        __builtin_mul_overflow(in, (long long)W, &in))
        return SV_ERR_INVALID_ARG;
    if (!aligned(parent, 4) || !aligned(lengths, 4)) return SV_ERR_MISALIGNED;
    const uintptr_t s0 = (uintptr_t)src, d0 = (uintptr_t)dst;
    if (s0 < d0 + (uintptr_t)out && d0 < s0 + (uintptr_t)in) return SV_ERR_INVALID_ARG;  // not in place
    ReorderArgs g = {};
    g.src = static_cast<const unsigned char*>(src);
    g.dst = static_cast<unsigned char*>(dst);
    g.parent = parent;
    g.lengths = lengths;
    g.S = S;
    g.tb = token_bytes;
    g.chunks = chunks;
    g.B = B;
    g.W = W;
    g.K = K;
    g.H = H;
    const uintptr_t bits = s0 | d0 | (uintptr_t)token_bytes;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = bits % 16 == 0 ? reorder<uint4>(g, st)
                          : bits % 4 == 0 ? reorder<uint32_t>(g, st)
                          : bits % 2 == 0 ? reorder<unsigned short>(g, st)
                                          : reorder<unsigned char>(g, st);
    return e == cudaSuccess ? SV_OK : (e == cudaErrorInvalidValue ? SV_ERR_INVALID_ARG : SV_ERR_CUDA);
}
