// Matrix product with bias, activation and residual in its epilogue: the projections around the
// layer. out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n], x and w in bf16 or
// fp16, products accumulated in fp32 on the tensor cores (tcgen05, TMEM), everything after them in
// fp32, one rounding to the output type.
// Pages: the input projections (qkvz, beta/alpha) and the output projection with the residual
// stream around build_layer_attn_linear_core (ik_llama.cpp src/llama-delta-net.cpp,
// build_layer_attn_linear), there plain ggml_mul_mat and ggml_add calls.
//
// linear_tile_kernel (up to about 128 tokens, and products with few output tiles): the weights are
// the M = 128 operand (128 output columns per CTA), the BM tokens of the tile the N operand, so
// that a single token pads the cheap side (16 rows of x) and the weights stream through shared
// memory once. Both operands are K-major 128-byte-swizzled tiles fetched by TMA through a ring that
// fills the SM's shared memory (the bytes in flight that HBM needs); rows and K elements beyond the
// arrays are filled with zeros by the TMA unit. When the output tiles alone would leave SMs idle,
// the CTAs of a cluster split K between them and join their fp32 partial sums through distributed
// shared memory, each CTA a share of the tokens, in rank order (deterministic, no workspace, no
// atomics).
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int LN_THREADS = 192;  // warps 0-3 epilogue (TMEM lanes 32 w ..), 4 TMA, 5 MMA
constexpr int LN_BN = 128;       // output columns per tile

struct LinearKernelArgs {
  const float* bias;
  const void* residual;
  void* out;
  int64_t M, ldr, ldo;
  int N, K;
  int act, res_dtype, out_dtype;  // res_dtype < 0: none
  int vec;                        // rows of out and residual allow vectors of 4 elements
  uint32_t idesc;
  int split;                      // CTAs per cluster, along K
  int32_t* status;
};

// ---------------------------------------------------------------- epilogue
// Activation, residual type and output type are template arguments of the row loops, chosen once
// per CTA: the loop that runs is a few dozen instructions (with the choices inside it, a tile's
// epilogue cost 8,000 to 45,000 cycles, most of them instruction fetch).
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == GDN_ACT_SILU) return silu_exact(v);
  if constexpr (ACT == GDN_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  if constexpr (ACT == GDN_ACT_SIGMOID) return sigmoidf_(v);
  return v;
}
struct NoResidual {};

// Rows r0, r0 + step, .. below `cnt` of a tile whose row 0 is output row m: 4 columns n .. n + 3 of
// each, from sums(row) -> float4. Four rows at a time, their residuals loaded together.
template <int ACT, typename TR, typename TO, typename Sums>
__device__ __forceinline__ void finish_rows(const LinearKernelArgs& p, int64_t m, int n, int r0,
                                            int step, int cnt, Sums sums) {
  if (n >= p.N) return;
  const int cols = p.N - n < 4 ? p.N - n : 4;
  float bias[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) bias[i] = p.bias && i < cols ? p.bias[n + i] : 0.f;
  TO* o = static_cast<TO*>(p.out) + (m + r0) * p.ldo + n;
  const int64_t ostep = p.ldo * step, rstep = p.ldr * step;
  if (p.vec && cols == 4) {
    const TR* res = nullptr;
    if constexpr (!std::is_same<TR, NoResidual>::value)
      res = static_cast<const TR*>(p.residual) + (m + r0) * p.ldr + n;
#pragma unroll 1
    for (int r = r0; r < cnt; r += 4 * step) {
      float4 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r + i * step < cnt) {
          if constexpr (!std::is_same<TR, NoResidual>::value) y[i] = ld4(res + i * rstep);
          x[i] = sums(r + i * step);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i * step < cnt)
          st4(o + i * ostep, make_float4(activate<ACT>(x[i].x + bias[0]) + y[i].x,
                                         activate<ACT>(x[i].y + bias[1]) + y[i].y,
                                         activate<ACT>(x[i].z + bias[2]) + y[i].z,
                                         activate<ACT>(x[i].w + bias[3]) + y[i].w));
      o += 4 * ostep;
      res += 4 * rstep;
    }
  } else {
    // odd strides, and the last columns of an N that is no multiple of 4
#pragma unroll 1
    for (int r = r0; r < cnt; r += step, o += ostep) {
      const float4 x4 = sums(r);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= cols) break;
        float v = activate<ACT>(x[i] + bias[i]);
        if constexpr (!std::is_same<TR, NoResidual>::value)
          v += ld(static_cast<const TR*>(p.residual) + (m + r) * p.ldr + n + i);
        st(o + i, v);
      }
    }
  }
}
template <int ACT, typename TR, typename Sums>
__device__ __forceinline__ void finish_o(const LinearKernelArgs& p, int64_t m, int n, int r0,
                                         int step, int cnt, Sums sums) {
  if (p.out_dtype == GDN_BF16) finish_rows<ACT, TR, __nv_bfloat16>(p, m, n, r0, step, cnt, sums);
  else if (p.out_dtype == GDN_F32) finish_rows<ACT, TR, float>(p, m, n, r0, step, cnt, sums);
  else finish_rows<ACT, TR, __half>(p, m, n, r0, step, cnt, sums);
}
template <int ACT, typename Sums>
__device__ __forceinline__ void finish_r(const LinearKernelArgs& p, int64_t m, int n, int r0,
                                         int step, int cnt, Sums sums) {
  if (p.res_dtype < 0) finish_o<ACT, NoResidual>(p, m, n, r0, step, cnt, sums);
  else if (p.res_dtype == GDN_BF16) finish_o<ACT, __nv_bfloat16>(p, m, n, r0, step, cnt, sums);
  else if (p.res_dtype == GDN_F32) finish_o<ACT, float>(p, m, n, r0, step, cnt, sums);
  else finish_o<ACT, __half>(p, m, n, r0, step, cnt, sums);
}
template <typename Sums>
__device__ __forceinline__ void finish(const LinearKernelArgs& p, int64_t m, int n, int r0, int step,
                                       int cnt, Sums sums) {
  if (p.act == GDN_ACT_NONE) finish_r<GDN_ACT_NONE>(p, m, n, r0, step, cnt, sums);
  else if (p.act == GDN_ACT_SILU) finish_r<GDN_ACT_SILU>(p, m, n, r0, step, cnt, sums);
  else if (p.act == GDN_ACT_GELU) finish_r<GDN_ACT_GELU>(p, m, n, r0, step, cnt, sums);
  else finish_r<GDN_ACT_SIGMOID>(p, m, n, r0, step, cnt, sums);
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in CTA `rank` of the cluster of what lies at `local` in this CTA.
__device__ __forceinline__ uint32_t at_rank(uint32_t local, uint32_t rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  return remote;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Arrive on a barrier of another CTA of the cluster, releasing this thread's (and, after
// __syncwarp, its warp's) earlier writes to it.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Wait on a barrier of this CTA that other CTAs arrive on (same limit as mbar_wait).
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > 2000000000LL) return false;
  }
}

// ---------------------------------------------------------------- tile kernel
// A stage holds LT_SUB(bm) sub-tiles of 64 K elements (one 128-byte swizzle row each) of both
// operands: two for up to 64 tokens, where a wait and its loop cost more than the four small MMAs
// of one sub-tile (350 against 160 to 190 cycles).
constexpr int lt_sub(int bm) { return bm == 32 || bm == 64 ? 2 : 1; }
constexpr int lt_stage(int bm) { return (LN_BN + bm) * 128 * lt_sub(bm); }
constexpr int lt_stages(int bm) { return bm <= 16 ? 5 : bm <= 32 ? 5 : bm <= 64 ? 4 : 5; }
constexpr int lt_sums(int bm) { return bm * LN_BN * 4; }  // the partial sums of the whole tile
constexpr int lt_smem(int bm) { return lt_stages(bm) * lt_stage(bm) + lt_sums(bm) + 1024; }

template <int BM>
__global__ void __launch_bounds__(LN_THREADS, 1)
linear_tile_kernel(const LinearKernelArgs p, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_x) {
  constexpr int NST = lt_stages(BM), SB = lt_stage(BM), SUB = lt_sub(BM), BK = 64 * SUB;
  constexpr uint32_t TCOLS = BM < 32 ? 32 : BM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  float* sums = reinterpret_cast<float*>(sm + NST * SB);  // [source rank][token][column]
  __shared__ uint64_t full[NST], empty[NST], done, joined;
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int split = p.split, rank = blockIdx.x % split;  // rank in the cluster (split, 1, 1)
  const int n0 = (blockIdx.x / split) * LN_BN;
  const int64_t m0 = (int64_t)blockIdx.y * BM;
  const int ksteps = (p.K + BK - 1) / BK;
  const int k0 = (int)((int64_t)ksteps * rank / split);
  const int nk = (int)((int64_t)ksteps * (rank + 1) / split) - k0;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(&done, 1);
    mbar_init(&joined, 4 * split);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&tmem_base, TCOLS);
    tmem_relinquish();  // at once: until then no other block is placed on this SM
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = tmem_base;
  if (split > 1) cluster_arrive();  // the barriers of this CTA are ready (waited for below)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 4) {
    if (elect_one()) {
      int i = 0;
      for (; i < nk; ++i) {
        const int st = i % NST;
        if (i >= NST && !mbar_wait(&empty[st], (i / NST - 1) & 1, &failed)) { failed = 1; break; }
        mbar_arrive_expect_tx(&full[st], SB);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
          tma_load_2d(sm + st * SB + u * LN_BN * 128, &tm_w, (k0 + i) * BK + u * 64, n0, &full[st]);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
          tma_load_2d(sm + st * SB + SUB * LN_BN * 128 + u * BM * 128, &tm_x,
                      (k0 + i) * BK + u * 64, (int)m0, &full[st]);
      }
      // after a time-out: no copy of this CTA may still be in flight when it ends
      if (i < nk)
        for (int j = i > NST ? i - NST : 0; j < i; ++j)
          mbar_wait(&full[j % NST], (j / NST) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      for (int i = 0; i < nk; ++i) {
        const int st = i % NST;
        if (!mbar_wait(&full[st], (i / NST) & 1, &failed)) { failed = 1; break; }
        fence_after_sync();
        const uint32_t a = smem_u32(sm + st * SB);
        const uint64_t da = desc_sw128(a, 16, 1024);
        const uint64_t db = desc_sw128(a + SUB * LN_BN * 128, 16, 1024);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 bytes along the swizzled row per K step
            mma_f16(tm, da + u * (LN_BN * 8) + 2 * k, db + u * (BM * 8) + 2 * k, p.idesc,
                    i > 0 || u > 0 || k > 0);
        commit(&empty[st]);
      }
      commit(&done);
    }
    __syncwarp();
  }
  // the accumulator is complete
  if (!mbar_wait(&done, 0, nullptr)) failed = 1;
  fence_after_sync();
  if (split > 1) cluster_wait();  // the other CTAs' barriers are ready

  // every token's partial sums to the rank that finishes it: rank r the tokens [r per, (r + 1) per)
  const int per = BM / split, per_log = 31 - __clz(per);
  if (warp < 4) {
    const int tokens = (int)(p.M - m0 < BM ? p.M - m0 : BM);
    const uint32_t mine = smem_u32(sums + rank * per * LN_BN + warp * 32 + lane);
    for (int c = 0; c < BM && c < tokens; c += 16) {
      uint32_t r[16];
      tmem_ld16(taddr(tm, warp * 32, c), r);
      tmem_wait_ld();
      if (split == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sums[(c + i) * LN_BN + warp * 32 + lane] = __uint_as_float(r[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st_cluster(at_rank(mine + (uint32_t)(((c + i) & (per - 1)) * LN_BN * 4), (c + i) >> per_log),
                     __uint_as_float(r[i]));
      }
    }
    if (split == 1) {
      asm volatile("bar.sync 1, 128;" ::: "memory");
    } else {
      __syncwarp();
      if (lane < split) arrive_cluster(at_rank(smem_u32(&joined), lane));
      if (!wait_cluster(&joined, 0)) failed = 1;
    }
    // each warp every fourth token of this rank's share, 4 columns per lane
    const int g = lane * 4;
    const int64_t mr = m0 + (int64_t)rank * per;
    const int cnt = p.M - mr < per ? (int)(p.M - mr) : per;
    if (!failed)
      finish(p, mr, n0 + g, warp, 4, cnt, [&](int t) {
        float4 v = *reinterpret_cast<const float4*>(sums + t * LN_BN + g);
        for (int s = 1; s < split; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(sums + (s * per + t) * LN_BN + g);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        return v;
      });
  }
  fence_before_sync();
  __syncthreads();
  if (failed && tid == 0) set_status(p.status, GDN_ETIMEOUT);
  if (warp == 5) tmem_dealloc(tm, TCOLS);
}

// ------------------------------------------------------------------------------- host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn linear_encode() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// 16-bit [rows][K] with a row stride of ld elements; box = 64 K elements x `box_rows` rows.
cudaError_t make_map(CUtensorMap* m, const void* base, bool bf16, int64_t rows, int K, int64_t ld,
                     int box_rows) {
  EncodeFn enc = linear_encode();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Vectors of 4 elements along the rows of an array: base and row stride are multiples of them.
bool rows_vec4(const void* p, int dtype, int64_t ld) {
  const size_t es = dtype == GDN_F32 ? 4 : 2;
  return (reinterpret_cast<uintptr_t>(p) & (4 * es - 1)) == 0 && ld % 4 == 0;
}
LinearKernelArgs kernel_args(const LinearArgs& a) {
  LinearKernelArgs k{};
  k.bias = a.bias; k.residual = a.residual; k.out = a.out;
  k.M = a.M; k.N = a.N; k.K = a.K; k.ldr = a.ldr; k.ldo = a.ldo;
  k.act = a.act; k.res_dtype = a.residual ? a.res_dtype : -1; k.out_dtype = a.out_dtype;
  k.vec = rows_vec4(a.out, a.out_dtype, a.ldo) &&
          (!a.residual || rows_vec4(a.residual, a.res_dtype, a.ldr));
  k.status = a.status;
  return k;
}

template <int BM>
cudaError_t launch_tile(const LinearArgs& a, int sms, cudaStream_t s) {
  const bool bf16 = a.dtype == GDN_BF16;
  alignas(64) CUtensorMap tm_w, tm_x;
  cudaError_t e = make_map(&tm_w, a.w, bf16, a.N, a.K, a.ldw, LN_BN);
  if (e == cudaSuccess) e = make_map(&tm_x, a.x, bf16, a.M, a.K, a.ldx, BM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_tile_kernel<BM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             lt_smem(BM));
  if (e != cudaSuccess) return e;
  const int64_t nt = (a.N + LN_BN - 1) / LN_BN, mt = (a.M + BM - 1) / BM;
  if (mt > 65535) return cudaErrorInvalidValue;
  // K split as far as the SMs hold the CTAs (one each), at least two stages for each
  const int ksteps = (a.K + 64 * lt_sub(BM) - 1) / (64 * lt_sub(BM));
  int split = 1;
  while (split < 8 && nt * mt * split * 2 <= sms && ksteps >= split * 2 * 2) split *= 2;
  LinearKernelArgs k = kernel_args(a);
  k.idesc = idesc_f16(LN_BN, BM, false, false) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
  k.split = split;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nt * split), (unsigned)mt);
  cfg.blockDim = dim3(LN_THREADS);
  cfg.dynamicSmemBytes = lt_smem(BM);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_tile_kernel<BM>, k, tm_w, tm_x);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (a.M <= 16) return launch_tile<16>(a, sms, s);
  if (a.M <= 32) return launch_tile<32>(a, sms, s);
  if (a.M <= 64) return launch_tile<64>(a, sms, s);
  return launch_tile<128>(a, sms, s);
}

}  // namespace gdn
