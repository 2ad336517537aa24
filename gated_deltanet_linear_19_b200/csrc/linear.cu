// Matrix product with bias, activation and residual in its epilogue: the projections around the
// layer. out[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + residual[m][n], x and w in bf16 or
// fp16, products accumulated in fp32 on the tensor cores (tcgen05, TMEM), everything after them in
// fp32, one rounding to the output type.
// Pages: the input projections (qkvz, beta/alpha) and the output projection with the residual
// stream around build_layer_attn_linear_core (ik_llama.cpp src/llama-delta-net.cpp,
// build_layer_attn_linear), there plain ggml_mul_mat and ggml_add calls.
//
// linear_tile_kernel: the weights are the M = 128 operand (128 output columns per CTA), the BM
// tokens of the tile the N operand, so that a single token pads the cheap side (16 rows of x) and
// the weights stream through shared memory once. Both operands are K-major 128-byte-swizzled tiles
// of 64 K elements fetched by TMA through a ring of stages; rows and K elements beyond the arrays
// are filled with zeros by the TMA unit. When the output tiles alone would leave SMs idle, the CTAs
// of a cluster split K between them and join their fp32 partial sums through distributed shared
// memory in rank order (deterministic, no workspace, no atomics).
#include <cuda.h>

#include <mutex>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int LN_THREADS = 192;  // warps 0-3 epilogue (TMEM lanes 32 w ..), 4 TMA, 5 MMA
constexpr int LN_BN = 128;       // output columns per tile
constexpr int LN_BK = 64;        // K elements per stage: one 128-byte swizzle row

struct LinearKernelArgs {
  const float* bias;
  const void* residual;
  void* out;
  int64_t M, ldr, ldo;
  int N, K;
  int act, res_dtype, out_dtype;  // res_dtype < 0: none
  uint32_t idesc;
  int split;                      // CTAs per cluster, along K
  int32_t* status;
};

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case GDN_ACT_SILU: return silu_exact(v);
    case GDN_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case GDN_ACT_SIGMOID: return sigmoidf_(v);
  }
  return v;
}
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == GDN_F32) return static_cast<const float*>(p)[i];
  if (dtype == GDN_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == GDN_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == GDN_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_remote(uint32_t local, uint32_t rank, float v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}

// Bytes of a stage, and stages such that two CTAs fit on an SM for up to 64 tokens.
constexpr int ln_stage_bytes(int bm) { return (LN_BN + bm) * LN_BK * 2; }
constexpr int ln_stages(int bm) { return bm <= 16 ? 6 : bm <= 32 ? 5 : bm <= 64 ? 4 : bm <= 128 ? 6 : 4; }
constexpr int ln_smem(int bm) { return ln_stages(bm) * ln_stage_bytes(bm) + 1024; }

// One finished column of the tile: 16 tokens m0.. of output column n.
__device__ __forceinline__ void finish16(const LinearKernelArgs& p, const float (&v)[16],
                                         int64_t m0, int n, float bias) {
  float r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    r[i] = (p.res_dtype >= 0 && m0 + i < p.M)
               ? load_any(p.residual, p.res_dtype, (m0 + i) * p.ldr + n) : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (m0 + i < p.M)
      store_any(p.out, p.out_dtype, (m0 + i) * p.ldo + n, activate(v[i] + bias, p.act) + r[i]);
}

template <int BM>
__global__ void __launch_bounds__(LN_THREADS)
linear_tile_kernel(const LinearKernelArgs p, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_x) {
  constexpr int NST = ln_stages(BM), SB = ln_stage_bytes(BM);
  constexpr uint32_t TCOLS = BM < 32 ? 32 : BM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[NST], empty[NST], done;
  __shared__ uint32_t tmem_base;
  __shared__ int failed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = p.split, rank = split > 1 ? (int)cluster_rank() : 0;
  const int n0 = (blockIdx.x / split) * LN_BN;
  const int64_t m0 = (int64_t)blockIdx.y * BM;
  const int ksteps = (p.K + LN_BK - 1) / LN_BK;
  const int k0 = (int)((int64_t)ksteps * rank / split);
  const int nk = (int)((int64_t)ksteps * (rank + 1) / split) - k0;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(&done, 1);
    failed = 0;
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc(&tmem_base, TCOLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == 4) {
    if (lane == 0) {
      int i = 0;
      for (; i < nk; ++i) {
        const int st = i % NST;
        if (i >= NST && !mbar_wait(&empty[st], (i / NST - 1) & 1, &failed)) { failed = 1; break; }
        mbar_arrive_expect_tx(&full[st], SB);
        tma_load_2d(sm + st * SB, &tm_w, (k0 + i) * LN_BK, n0, &full[st]);
        tma_load_2d(sm + st * SB + LN_BN * LN_BK * 2, &tm_x, (k0 + i) * LN_BK, (int)m0, &full[st]);
      }
      // after a time-out: no copy of this CTA may still be in flight when it ends
      if (failed)
        for (int j = i > NST ? i - NST : 0; j < i; ++j) mbar_wait(&full[j % NST], (j / NST) & 1, nullptr);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      for (int i = 0; i < nk; ++i) {
        const int st = i % NST;
        if (!mbar_wait(&full[st], (i / NST) & 1, &failed)) { failed = 1; break; }
        fence_after_sync();
        const uint32_t a = smem_u32(sm + st * SB), b = a + LN_BN * LN_BK * 2;
#pragma unroll
        for (int k = 0; k < LN_BK / 16; ++k)
          mma_f16(tm, desc_sw128(a + k * 32, 16, 1024), desc_sw128(b + k * 32, 16, 1024), p.idesc,
                  i > 0 || k > 0);
        commit(&empty[st]);
      }
      commit(&done);
    }
    __syncwarp();
  }
  // the accumulator is complete (and, with it, every copy and every read of the stages)
  if (!mbar_wait(&done, 0, nullptr)) failed = 1;
  fence_after_sync();
  __syncthreads();
  if (failed && tid == 0) set_status(p.status, GDN_ETIMEOUT);

  const int n = n0 + warp * 32 + lane;  // warps 0-3
  const float bias = (warp < 4 && p.bias && n < p.N) ? p.bias[n] : 0.f;
  if (split == 1) {
    if (warp < 4) {
      for (int c = 0; c < BM && m0 + c < p.M; c += 16) {
        uint32_t r[16];
        tmem_ld16(taddr(tm, warp * 32, c), r);
        tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
        if (n < p.N && !failed) finish16(p, v, m0 + c, n, bias);
      }
    }
  } else {
    // rank r joins the tokens [r BM / split, ..) of the tile: the others' partial sums come into
    // its stage memory as [source rank][token][column]
    const int per = BM / split;
    float* recv = reinterpret_cast<float*>(sm);
    cluster_sync();  // every CTA of the cluster has finished reading its stages
    if (warp < 4) {
      for (int c = 0; c < BM && m0 + c < p.M; c += 16) {
        uint32_t r[16];
        tmem_ld16(taddr(tm, warp * 32, c), r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int to = (c + i) / per, ml = (c + i) % per;
          st_remote(smem_u32(recv + ((rank * per + ml) * LN_BN) + warp * 32 + lane), to,
                    __uint_as_float(r[i]));
        }
      }
    }
    cluster_sync();
    if (warp < 4 && n < p.N && !failed) {
      for (int c = 0; c < per; c += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i] = 0.f;
          if (c + i < per)
            for (int s = 0; s < split; ++s)
              v[i] += recv[(s * per + c + i) * LN_BN + warp * 32 + lane];
        }
        // tokens beyond this rank's share belong to the next rank
        LinearKernelArgs q = p;
        const int64_t end = m0 + (int64_t)(rank + 1) * per;
        q.M = end < p.M ? end : p.M;
        finish16(q, v, m0 + (int64_t)rank * per + c, n, bias);
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tmem_relinquish();
    tmem_dealloc(tm, TCOLS);
  }
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
  const cuuint32_t box[2] = {LN_BK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BM>
cudaError_t launch_tile(const LinearArgs& a, int sms, cudaStream_t s) {
  const bool bf16 = a.dtype == GDN_BF16;
  alignas(64) CUtensorMap tm_w, tm_x;
  cudaError_t e = make_map(&tm_w, a.w, bf16, a.N, a.K, a.ldw, LN_BN);
  if (e == cudaSuccess) e = make_map(&tm_x, a.x, bf16, a.M, a.K, a.ldx, BM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(linear_tile_kernel<BM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ln_smem(BM));
  if (e != cudaSuccess) return e;
  const int64_t nt = (a.N + LN_BN - 1) / LN_BN, mt = (a.M + BM - 1) / BM;
  if (mt > 65535) return cudaErrorInvalidValue;
  const int ksteps = (a.K + LN_BK - 1) / LN_BK;
  const int64_t room = (BM <= 64 ? 2 : 1) * (int64_t)sms;  // CTAs resident at once
  int split = 1;
  while (split < 8 && nt * mt * split * 2 <= room && ksteps >= split * 2 * 4) split *= 2;
  LinearKernelArgs k{};
  k.bias = a.bias; k.residual = a.residual; k.out = a.out;
  k.M = a.M; k.N = a.N; k.K = a.K; k.ldr = a.ldr; k.ldo = a.ldo;
  k.act = a.act; k.res_dtype = a.residual ? a.res_dtype : -1; k.out_dtype = a.out_dtype;
  k.idesc = idesc_f16(LN_BN, BM, false, false) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
  k.split = split;
  k.status = a.status;
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
  cfg.dynamicSmemBytes = ln_smem(BM);
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
  if (a.M <= 128) return launch_tile<128>(a, sms, s);
  return launch_tile<256>(a, sms, s);
}

}  // namespace gdn
