// Draft step with rollback: a few drafted tokens per sequence (speculative decoding) run from the
// committed state without advancing it, and what a later commit needs of them is recorded, so
// that a rejected token costs nothing to undo.
// Pages: the per-token step of qwen3next.cpp build_delta_net_autoregressive
// (S <- exp(g) S; u = beta (v - S^T k); S <- S + k u^T; o = S^T q); the pages have no rollback.
//
// With e_i = exp(g_i), D_ij = prod_{l=j+1..i} e_l and c_i = prod_{l<=i} e_l, the drafted tokens
// i = 0..T-1 from state S are
//   u_i = beta_i (v_i - c_i S^T k_i - sum_{j<i} D_ij (k_i.k_j) u_j)
//   o_i = c_i S^T q_i + sum_{j<=i} D_ij (q_i.k_j) u_j
// and committing the first a tokens of a record is
//   S <- (prod_{l<a} e_l) S + sum_{j<a} (prod_{l=j+1..a-1} e_l) k_j u_j^T,
// which is the token recurrence unrolled: no token waits for the state update of the one before,
// so the state is read once, written at most once (only when something is committed), and the
// column sums S^T [k, q] of all tokens come from one pass over it. The decays are running
// products of numbers exp(g), never differences of cumulative logarithms, so gates of any size
// (down to -inf) lose nothing. fp32 throughout: o, u and the state equal the token recurrence to
// fp32 rounding.
//
// Two kernels, the second launched programmatically on the first:
//  - draft_prep_kernel, one block per (key head, sequence): validity of the sequence; q and k
//    (given, or from raw x: conv from the window behind the accepted tokens, SiLU, L2 norm), the
//    gates, the tokens' dot products and the two T x T coefficient tables, the accepted keys of
//    the old record and then the new record's keys, decays and inputs. What the second kernel
//    needs goes to the workspace (a few KB per head, read from L2).
//  - draft_state_kernel, HBM-bound, over tiles of up to 64 columns of one (value head, sequence):
//    commit, column sums, the T-step triangular solve per column, o and the record's u. As many
//    blocks as fit stay resident and take tiles in turn. A tile's inputs come by asynchronous
//    copies (TMA for the state, bulk copies for the rest) that are started when the block has
//    moved the tile before into registers, so that HBM works while the block computes; the first
//    tile's state is asked for before the first kernel has finished.
// The keys of a record are shared by the column tiles and value heads of a key head, so they are
// rewritten by the first kernel, which alone reads them; u belongs to one tile; the count n is
// read by the first kernel and written by the second. Nothing is read and written by different
// blocks of one kernel.
#include <cuda.h>

#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int DR_THREADS = 128;
constexpr int DR_MAX = 16;  // tokens per draft, at most
// Per (sequence, value head) in the workspace, for T tokens padded to TT = token_pad(T):
// Lt[TT][TT] with Lt[j][i] = beta_i D_ij (k_i.k_j) (j < i), P[TT][TT] with P[i][j] = D_ij (q_i.k_j)
// (j <= i), zeros elsewhere; c[TT], beta[TT]; the commit weights of the accepted tokens [DR_MAX]
// and that of the old state.
__host__ __device__ __forceinline__ int token_pad(int T) { return T <= 4 ? 4 : T <= 8 ? 8 : 16; }
__host__ __device__ __forceinline__ int coef_size(int T) {
  const int tt = token_pad(T);
  return 2 * tt * tt + 2 * tt + DR_MAX + 4;
}
constexpr int DR_COEF = 2 * DR_MAX * DR_MAX + 3 * DR_MAX + 4;  // coef_size(DR_MAX)

// Bytes of state that the first kernel asks L2 for ahead of the second: about what HBM delivers
// while it runs.
constexpr int64_t kStateAhead = 32 << 20;

// A set of the state kernel's second inputs in shared memory (es: bytes of a v element), in floats.
__host__ __device__ __forceinline__ int late_floats(int d_k, int ct, int depth, int es) {
  return 2 * depth * d_k + coef_size(depth) + depth * ct * es / 4;
}

// What the first kernel decides about a sequence.
struct alignas(16) DraftHeader {
  int run;   // 0: skipped (invalid); 1: processed
  int acc;   // accepted tokens of the old record
  int len;   // new tokens
  int rst;   // starts from a zero state
  int slot;
  int c0;    // first new token
  int pad0, pad1;
};

// x += k s over a quad of columns.
__device__ __forceinline__ void fma_row(float* x, const float4& s, float k) {
  x[0] = fmaf(s.x, k, x[0]);
  x[1] = fmaf(s.y, k, x[1]);
  x[2] = fmaf(s.z, k, x[2]);
  x[3] = fmaf(s.w, k, x[3]);
}

// N consecutive floats (N a power of two) from shared memory.
template <int N>
__device__ __forceinline__ void load_rows(float* x, const float* from) {
  if constexpr (N == 1) {
    x[0] = from[0];
  } else if constexpr (N == 2) {
    const float2 a = *reinterpret_cast<const float2*>(from);
    x[0] = a.x; x[1] = a.y;
  } else {
#pragma unroll
    for (int m = 0; m < N; m += 4) {
      const float4 a = *reinterpret_cast<const float4*>(from + m);
      x[m] = a.x; x[m + 1] = a.y; x[m + 2] = a.z; x[m + 3] = a.w;
    }
  }
}

struct DraftWs {
  size_t hdr, qk, rk, coef, v, o32, total;
};
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
DraftWs draft_ws(int H_k, int H_v, int d_k, int d_v, int64_t T, int n_seqs, int depth) {
  DraftWs w{};
  const size_t nk = (size_t)n_seqs * H_k, nv = (size_t)n_seqs * H_v;
  w.hdr = 0;
  w.qk = up256((size_t)n_seqs * sizeof(DraftHeader));
  w.rk = w.qk + up256(nk * 2 * depth * d_k * 4);
  w.coef = w.rk + up256(nk * depth * d_k * 4);
  w.v = w.coef + up256(nv * DR_COEF * 4);
  w.o32 = w.v + up256((size_t)T * H_v * d_v * 4);
  w.total = w.o32 + up256((size_t)T * H_v * d_v * 4);
  return w;
}

// The dot products of NT4 = 4 BS padded tokens: rows 0..NT4-1 of `vec` are k, rows NT4.. are q,
// all against the k rows. Every warp takes a quarter of the DK dimensions; a lane holds BS x BS
// outputs, of rows ib + 8 a and columns jb + 4 b (interleaved so that the eight row addresses of
// a load fall into different banks). Partial sums of the 4 warps go to part[warp][row][col].
template <int BS, int DK>
__device__ __forceinline__ void token_dots(const float* vec, float* part) {
  constexpr int LDV = DK + 4, QPW = DK / 16;  // float4 groups per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ib = lane >> 2, jb = lane & 3;
  float acc[BS][BS];
#pragma unroll
  for (int a = 0; a < BS; ++a)
#pragma unroll
    for (int b = 0; b < BS; ++b) acc[a][b] = 0.f;
#pragma unroll
  for (int g = 0; g < QPW; ++g) {
    const int d = (warp * QPW + g) * 4;
    float4 x[BS], y[BS];
#pragma unroll
    for (int a = 0; a < BS; ++a) {
      x[a] = *reinterpret_cast<const float4*>(vec + (ib + 8 * a) * LDV + d);
      y[a] = *reinterpret_cast<const float4*>(vec + (jb + 4 * a) * LDV + d);
    }
#pragma unroll
    for (int a = 0; a < BS; ++a)
#pragma unroll
      for (int b = 0; b < BS; ++b) {
        acc[a][b] = fmaf(x[a].x, y[b].x, acc[a][b]);
        acc[a][b] = fmaf(x[a].y, y[b].y, acc[a][b]);
        acc[a][b] = fmaf(x[a].z, y[b].z, acc[a][b]);
        acc[a][b] = fmaf(x[a].w, y[b].w, acc[a][b]);
      }
  }
#pragma unroll
  for (int a = 0; a < BS; ++a)
#pragma unroll
    for (int b = 0; b < BS; ++b)
      part[(warp * 8 * BS + ib + 8 * a) * 4 * BS + jb + 4 * b] = acc[a][b];
}

// TX: q, k (given) or x; TS: conv state. FUSED: from raw x.
template <int DK, typename TX, typename TS, bool FUSED>
__global__ void __launch_bounds__(DR_THREADS, FUSED ? 4 : 7) draft_prep_kernel(const DraftArgs p) {
  constexpr int LDV = DK + 4, LPH = DK / 4;
  extern __shared__ __align__(128) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x, n = blockIdx.y;
  const int r = p.H_v / p.H_k, D = p.rec.depth;
  const bool lead = tid == 0 && hk == 0;
  // the kernels before have ended when the second kernel's blocks start
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  DraftHeader* hdr = reinterpret_cast<DraftHeader*>(ws + p.ws_hdr) + n;

  // ---- validity (the same decision in every block of the sequence); what needs one more load,
  // the record's count, and the earlier slot ids are looked at while the inputs are on their way
  const int64_t c0 = cu_at(p.cu_seqlens, n), c1 = cu_at(p.cu_seqlens, n + 1);
  const int slot = p.slot_ids[n];
  const bool rst = p.reset != nullptr && p.reset[n] != 0;
  const int acc_in = (rst || !p.accepted) ? 0 : p.accepted[n];
  int err = 0;
  if (c0 < 0 || c1 < c0 || c1 > p.T_total || c1 - c0 > D) err = GDN_EINVAL;
  else if (slot < 0 || slot >= p.n_slots) err = GDN_ESLOT;
  const bool known = err == 0 && acc_in >= 0 && acc_in <= D;
  const int T = known ? (int)(c1 - c0) : 0, acc = known ? acc_in : 0;
  const int most = acc_in != 0 && err == 0 ? p.rec.n[slot] : 0;
  // The second kernel's state stream starts here: the first blocks of the grid, whose states are
  // the first to be used, ask L2 for them (kStateAhead).
  if (tid < r && (T > 0 || acc > 0) && !rst && n * p.H_k + hk < p.pf_blocks) {
    const int h = (p.layout & GDN_GQA_TILED) ? hk + tid * p.H_k : hk * r + tid;
    prefetch_l2(p.state + ((int64_t)slot * p.H_v + h) * DK * p.d_v, (uint32_t)(DK * p.d_v * 4));
  }
  int hit = 0;
  for (int m = tid; m < n; m += DR_THREADS) hit |= p.slot_ids[m] == slot;
  // Settles the validity (block-wide): false, and the error on record, for a sequence to skip.
  auto settle = [&]() {
    if (__syncthreads_or(hit) && err == 0) err = GDN_ESLOT;
    if (err == 0 && acc_in != 0 && (acc_in < 0 || acc_in > D || acc_in > most)) err = GDN_EINVAL;
    if (lead) {
      if (err != 0) set_status(p.status, err);
      *hdr = err != 0 ? DraftHeader{} : DraftHeader{1, acc, T, rst ? 1 : 0, slot, (int)c0, 0, 0};
    }
    return err == 0;
  };
  const int T4 = token_pad(T), TD = token_pad(D);

  float* vec = sm;                     // [2 T4][LDV]: k rows 0..T4-1, q rows T4..2 T4-1
  float* part = vec + 2 * TD * LDV;    // [4][2 T4][T4]
  float* ge = part + 4 * 2 * TD * TD;  // [r][DR_MAX] new decays
  float* gb = ge + r * DR_MAX;         // [r][DR_MAX] new betas
  float* go = gb + r * DR_MAX;         // [r][DR_MAX] old decays

  if constexpr (!FUSED) {
    for (int i = tid; i < 2 * T * LPH; i += DR_THREADS) {
      const int w = i / (T * LPH), t = i / LPH - w * T, d = (i % LPH) * 4;
      const TX* src = static_cast<const TX*>(w ? p.q : p.k) + ((c0 + t) * p.H_k + hk) * DK + d;
      *reinterpret_cast<float4*>(vec + (w * T4 + t) * LDV + d) = ld4(src);
    }
    if (!settle()) return;
  }

  // The accepted keys of the old record, to the workspace; the thread that reads an element here is
  // the one that overwrites it below.
  float* rk = reinterpret_cast<float*>(ws + p.ws_rk) + ((int64_t)n * p.H_k + hk) * D * DK;
  float* reck = p.rec.k + ((int64_t)slot * p.H_k + hk) * D * DK;
  auto keep_keys = [&]() {
    for (int i = tid; i < acc * LPH; i += DR_THREADS)
      reinterpret_cast<float4*>(rk)[i] = reinterpret_cast<const float4*>(reck)[i];
  };
  // Gates of the key head's value heads, old and new decays.
  auto gates = [&]() {
    for (int i = tid; i < r * DR_MAX; i += DR_THREADS) {
      const int jv = i / DR_MAX, t = i % DR_MAX;
      const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
      float* rece = p.rec.e + ((int64_t)slot * p.H_v + h) * D;
      if (t < acc) go[i] = rece[t];
      if (t < T) {
        float e, b;
        if constexpr (FUSED) {
          const float z = gate_alpha(p.fa, c0 + t, h, p.H_k, p.H_v, p.layout) + p.dt_bias[h];
          e = expf(-expf(p.A_log[h]) * softplusf_(z));
          b = sigmoidf_(gate_beta_logit(p.fa, p.fb, c0 + t, h, p.H_k, p.H_v, p.layout));
        } else {
          e = expf(p.g[(c0 + t) * p.H_v + h]);
          b = p.beta[(c0 + t) * p.H_v + h];
        }
        ge[i] = e;
        gb[i] = b;
        rece[t] = e;
      }
    }
  };

  // ---- q and k of the tokens into shared memory and v to the workspace, from raw x
  if constexpr (FUSED) {
    const int R = p.d_conv > 0 ? p.d_conv - 1 : 0;
    const int64_t conv_dim = 2LL * p.H_k * DK + (int64_t)p.H_v * p.d_v;
    TS* cst = R > 0 ? static_cast<TS*>(p.conv_state) + (int64_t)slot * R * conv_dim : nullptr;
    TS* recx = R > 0 ? static_cast<TS*>(p.rec.x) + (int64_t)slot * D * conv_dim : nullptr;
    const TX* xg = static_cast<const TX*>(p.x);
    float* vg = reinterpret_cast<float*>(ws + p.ws_v);
    const int vq = p.d_v / 4;
    // warp 0: q, warp 1: k, warps 2 and 3: the v quads of the r value heads
    const int n_item = warp < 2 ? 1 : (r * vq + 63 - (tid - 64)) / 64;
    bool settled = false;
    for (int it = 0; it < n_item || !settled; ++it) {
      int64_t ch = 0;
      bool active = it < n_item;
      int jv = 0, qd = 0;
      if (warp < 2) {
        active = active && lane < LPH;
        if (active) ch = (int64_t)warp * p.H_k * DK + (int64_t)hk * DK + lane * 4;
      } else if (active) {
        const int item = tid - 64 + it * 64;
        jv = item / vq; qd = item % vq;
        const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
        ch = 2LL * p.H_k * DK + (int64_t)h * p.d_v + qd * 4;
      }
      // taps right-aligned: wa[.][3] multiplies the current token, wa[.][2 - i] the window
      float wa[4][4], win[3][4];
      if (p.d_conv == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 w = active ? ld4(p.conv_w + (ch + j) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
          wa[j][0] = w.x; wa[j][1] = w.y; wa[j][2] = w.z; wa[j][3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tap = p.d_conv - 4 + i;
            wa[j][i] = (active && tap >= 0) ? p.conv_w[(ch + j) * p.d_conv + tap] : 0.f;
          }
      }
      // the window behind the accepted tokens: the last R rows of [conv state; recorded x[:acc]]
#pragma unroll
      for (int sl = 0; sl < 3; ++sl) {
        const int row = sl - (3 - R);  // 0 = oldest
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (active && row >= 0 && !rst && known) {
          const int at = row + acc;
          v = at < R ? ld4(cst + (int64_t)at * conv_dim + ch)
                     : ld4(recx + (int64_t)(at - R) * conv_dim + ch);
        }
        win[sl][0] = v.x; win[sl][1] = v.y; win[sl][2] = v.z; win[sl][3] = v.w;
      }
      float4 xr[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        xr[u] = (active && u < T) ? ld4(xg + (c0 + u) * conv_dim + ch)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      if (!settled) {
        settled = true;
        if (!settle()) return;
        keep_keys();
        gates();
      }
      if (active && R > 0 && (acc > 0 || rst)) {
#pragma unroll
        for (int sl = 0; sl < 3; ++sl) {
          const int row = sl - (3 - R);
          if (row >= 0)
            st4(cst + (int64_t)row * conv_dim + ch,
                make_float4(win[sl][0], win[sl][1], win[sl][2], win[sl][3]));
        }
      }
      for (int tb = 0; tb < T; tb += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = tb + u;
          if (t >= T) break;
          const float xs[4] = {xr[u].x, xr[u].y, xr[u].z, xr[u].w};
          if (active && R > 0) st4(recx + (int64_t)t * conv_dim + ch, xr[u]);
          float y[4], ss = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (p.d_conv > 0) {
              float a = wa[j][0] * win[0][j];
              a = fmaf(wa[j][1], win[1][j], a);
              a = fmaf(wa[j][2], win[2][j], a);
              a = fmaf(wa[j][3], xs[j], a);
              y[j] = a * sigmoidf_(a);
            } else {
              y[j] = xs[j];
            }
            ss = fmaf(y[j], y[j], ss);
            win[0][j] = win[1][j];
            win[1][j] = win[2][j];
            win[2][j] = xs[j];
          }
          // the next four tokens' inputs are asked for as these are used
          if (active && t + 4 < T) xr[u] = ld4(xg + (c0 + t + 4) * conv_dim + ch);
          if (warp < 2) {
            const float mul = (warp == 0 ? p.q_scale : 1.0f) / sqrtf(warp_sum(ss) + p.eps);
            if (active)
              *reinterpret_cast<float4*>(vec + ((warp == 0 ? T4 : 0) + t) * LDV + lane * 4) =
                  make_float4(y[0] * mul, y[1] * mul, y[2] * mul, y[3] * mul);
          } else if (active) {
            const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
            *reinterpret_cast<float4*>(vg + ((c0 + t) * p.H_v + h) * p.d_v + qd * 4) =
                make_float4(y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
  } else {
    keep_keys();
    gates();
  }
  __syncthreads();

  // ---- the new record's keys, and q and k for the state kernel
  float* qk = reinterpret_cast<float*>(ws + p.ws_qk) + ((int64_t)n * p.H_k + hk) * 2 * D * DK;
  for (int i = tid; i < T * LPH; i += DR_THREADS) {
    const int t = i / LPH, d = (i % LPH) * 4;
    const float4 kv = *reinterpret_cast<const float4*>(vec + t * LDV + d);
    reinterpret_cast<float4*>(reck)[i] = kv;
    reinterpret_cast<float4*>(qk)[i] = kv;
    *reinterpret_cast<float4*>(qk + (int64_t)T * DK + i * 4) =
        *reinterpret_cast<const float4*>(vec + (T4 + t) * LDV + d);
  }

  // ---- dot products (rows T..T4-1 are never read back), then the coefficient tables
  if (T4 == 4) token_dots<1, DK>(vec, part);
  else if (T4 == 8) token_dots<2, DK>(vec, part);
  else token_dots<4, DK>(vec, part);
  __syncthreads();
  float* coef = reinterpret_cast<float*>(ws + p.ws_coef);
  for (int i = tid; i < r * T4 * T4; i += DR_THREADS) {
    const int jv = i / (T4 * T4), row = (i / T4) % T4, col = i % T4;
    const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
    float* cL = coef + ((int64_t)n * p.H_v + h) * DR_COEF;
    float* cP = cL + T4 * T4;
    float* cC = cP + T4 * T4;
    const bool in = row < T && col <= row;
    float d = 1.f, kk = 0.f, qq = 0.f;
    if (in) {
      for (int l = col + 1; l <= row; ++l) d *= ge[jv * DR_MAX + l];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        kk += part[(w * 2 * T4 + row) * T4 + col];
        qq += part[(w * 2 * T4 + T4 + row) * T4 + col];
      }
    }
    cP[row * T4 + col] = in ? d * qq : 0.f;
    cL[col * T4 + row] = in && col < row ? gb[jv * DR_MAX + row] * d * kk : 0.f;
    if (row == 0 && col < T) {
      float c = 1.f;
      for (int l = 0; l <= col; ++l) c *= ge[jv * DR_MAX + l];
      cC[col] = c;
      cC[T4 + col] = gb[jv * DR_MAX + col];
    }
  }
  for (int i = tid; i < r * acc; i += DR_THREADS) {
    const int jv = i / acc, j = i - jv * acc;
    const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
    float* cW = coef + ((int64_t)n * p.H_v + h) * DR_COEF + 2 * T4 * T4 + 2 * T4;
    float w = 1.f;
    for (int l = j + 1; l < acc; ++l) w *= go[jv * DR_MAX + l];
    cW[j] = w;
    if (j == 0) cW[DR_MAX] = w * go[jv * DR_MAX];
  }
}

// One (column tile, value head, sequence) of the state kernel's work.
struct DraftTile {
  int n, h, ct;  // sequence, value head, column tile
  bool loaded;   // its copies are under way
  DraftHeader hd;
};
__device__ __forceinline__ DraftTile tile_at(const DraftArgs& p, unsigned t, int tiles_c) {
  const unsigned per = (unsigned)(p.H_v * tiles_c);
  DraftTile w;
  w.n = (int)(t / per);
  const unsigned rem = t - (unsigned)w.n * per;
  w.h = (int)(rem / (unsigned)tiles_c);
  w.ct = (int)(rem - (unsigned)w.h * (unsigned)tiles_c);
  return w;
}
__device__ __forceinline__ DraftHeader header_at(const DraftArgs& p, int n) {
  const int4* g = reinterpret_cast<const int4*>(static_cast<const uint8_t*>(p.workspace) + p.ws_hdr) +
                  2 * (int64_t)n;
  const int4 a = g[0], b = g[1];
  return DraftHeader{a.x, a.y, a.z, a.w, b.x, b.y, 0, 0};
}
// A sequence without accepted and without new tokens needs no state, unless it starts from zero.
__device__ __forceinline__ bool tile_works(const DraftHeader& h) {
  return h.run && (h.acc > 0 || h.len > 0 || h.rst);
}

// Threads of a block of the state kernel and, at most, blocks of it on an SM, for records of up to
// max_t tokens: 16 warps on an SM either way, but the longer records' inputs leave shared memory
// for two blocks only.
__host__ __device__ constexpr int st_threads(int max_t) { return max_t <= 8 ? 128 : 256; }
__host__ __device__ constexpr int st_blocks(int max_t) { return max_t <= 8 ? 4 : 2; }
constexpr int ST_GROUP = 4;  // tokens summed between two barriers

template <int DK, int CT, int MAXT>
__global__ void __launch_bounds__(st_threads(MAXT), st_blocks(MAXT))
    draft_state_kernel(const DraftArgs p, const __grid_constant__ CUtensorMap tm_state) {
  constexpr int NT = st_threads(MAXT), NW = NT / 32;
  constexpr int RPT = DK * CT / (4 * NT);    // state rows of a thread
  constexpr int QL = CT / 4, NRW = 32 / QL;  // lanes per row, row groups of a warp
  constexpr int TEAMS = NT / CT;             // threads per column behind the sums
  constexpr int G = ST_GROUP;
  static_assert(RPT >= 1 && MAXT % TEAMS == 0, "shape");
  extern __shared__ __align__(128) float sm[];
  __shared__ __align__(8) uint64_t full;
  __shared__ DraftTile tiles[2];  // this tile and the next
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cq = tid % QL, row0 = (tid / QL) * RPT;
  const int D = p.rec.depth, d_v = p.d_v, tiles_c = d_v / CT;
  const unsigned total = (unsigned)p.n_seqs * (unsigned)(p.H_v * tiles_c);
  const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
  const int es = p.qkv_dtype == GDN_F32 ? 4 : 2;

  float* st_s = sm;               // [DK][CT] state
  float* rk_s = st_s + DK * CT;   // [D][DK] accepted keys
  float* uo_s = rk_s + D * DK;    // [D][CT] their u
  // two sets of: keys and queries [2][T][DK], coefficients, v [T][CT] in its own type. Rows up to
  // the next multiple of 4 tokens are read (what they give is dropped): at most 3 DK floats behind
  // the last set's queries, all inside this block's memory.
  float* late = uo_s + D * CT;
  const int late_sz = late_floats(DK, CT, D, es);
  float* red = late + 2 * late_sz;   // [warps][k, q][G][CT]
  float* w_s = red + 2 * NW * G * CT;  // [MAXT][CT] right-hand sides of u

  // Loads of a tile, by warp 0: the state (unless the first tile has asked for it already) and
  // the rest of what its sequence needs, all counted on `full`.
  auto load_tile = [&](const DraftTile& w, int set, bool with_state) {
    const int T = w.hd.len, acc = w.hd.acc;
    float* qk = late + set * late_sz;
    float* cf = qk + 2 * D * DK;
    uint8_t* vs = reinterpret_cast<uint8_t*>(cf + coef_size(D));
    const int cbytes = coef_size(T) * 4;
    if (lane == 0) {
      umma::mbar_arrive_expect_tx(&full, (uint32_t)((with_state ? DK * CT * 4 : 0) +
                                                    acc * (DK + CT) * 4 + 2 * T * DK * 4 + cbytes +
                                                    T * CT * es));
    }
    __syncwarp();
    const int hk = khead_of(w.h, p.H_k, p.H_v, p.layout);
    const int64_t nk = (int64_t)w.n * p.H_k + hk;
    if (lane == 0 && with_state)
      umma::tma_load_3d(st_s, &tm_state, w.ct * CT, 0, w.hd.slot * p.H_v + w.h, &full);
    if (lane == 1 && acc > 0)
      umma::bulk_g2s(rk_s, reinterpret_cast<const float*>(ws + p.ws_rk) + nk * D * DK, acc * DK * 4,
                     &full);
    if (lane == 2 && T > 0)
      umma::bulk_g2s(qk, reinterpret_cast<const float*>(ws + p.ws_qk) + nk * 2 * D * DK,
                     2 * T * DK * 4, &full);
    if (lane == 3)
      umma::bulk_g2s(cf, reinterpret_cast<const float*>(ws + p.ws_coef) +
                             ((int64_t)w.n * p.H_v + w.h) * DR_COEF, cbytes, &full);
    if (lane < acc)
      umma::bulk_g2s(uo_s + lane * CT,
                     p.rec.u + (((int64_t)w.hd.slot * p.H_v + w.h) * D + lane) * d_v + w.ct * CT,
                     CT * 4, &full);
    if (lane >= 16 && lane - 16 < T)
      umma::bulk_g2s(vs + (lane - 16) * CT * es,
                     static_cast<const uint8_t*>(p.v) +
                         (((int64_t)(w.hd.c0 + lane - 16) * p.H_v + w.h) * d_v + w.ct * CT) * es,
                     CT * es, &full);
  };

  // ---- the first tile's state, before the first kernel's decision on its sequence is known (the
  // state was written before that kernel started)
  unsigned t = blockIdx.x;
  if (tid == 0) {
    umma::mbar_init(&full, 1);
    umma::fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    DraftTile w = tile_at(p, t, tiles_c);
    const int slot = p.slot_ids[w.n];
    const bool rst = p.reset != nullptr && p.reset[w.n] != 0;
    const bool idle = cu_at(p.cu_seqlens, w.n + 1) == cu_at(p.cu_seqlens, w.n) &&
                      (!p.accepted || p.accepted[w.n] == 0);
    const bool early = slot >= 0 && slot < p.n_slots && !rst && !idle;
    if (early && lane == 0) {
      umma::mbar_expect_tx(&full, DK * CT * 4);
      umma::tma_load_3d(st_s, &tm_state, w.ct * CT, 0, slot * p.H_v + w.h, &full);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // what the first kernel wrote is read by bulk copies too
    asm volatile("fence.proxy.async.global;" ::: "memory");
    w.hd = header_at(p, w.n);
    w.loaded = early || tile_works(w.hd);
    if (tile_works(w.hd)) load_tile(w, 0, !early && !w.hd.rst);
    else if (early && lane == 0) umma::mbar_arrive(&full);
    if (lane == 0) tiles[0] = w;
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  __syncthreads();

  uint32_t phase = 0;
  for (int it = 0;; ++it, t += gridDim.x) {
    const bool more = t + gridDim.x < total;
    if (more && warp == 0) {
      DraftTile w = tile_at(p, t + gridDim.x, tiles_c);
      w.hd = header_at(p, w.n);
      w.loaded = tile_works(w.hd);
      if (lane == 0) tiles[(it + 1) & 1] = w;
    }
    const DraftTile& cur = tiles[it & 1];
    const int T = cur.hd.len, acc = cur.hd.acc;
    const bool rst = cur.hd.rst != 0, works = tile_works(cur.hd);
    float* qk_s = late + (it & 1) * late_sz;
    const float* cf = qk_s + 2 * D * DK;
    const int TT = token_pad(T);
    const float* cL = cf;                   // [TT][TT]: Lt[j][i]
    const float* cP = cL + TT * TT;         // [TT][TT]: P[i][j]
    const float* cC = cP + TT * TT;
    const float* cB = cC + TT;
    const float* cW = cB + TT;              // commit weights, then that of the old state
    float4 s[RPT];
    if (cur.loaded) {
      if (!umma::mbar_wait(&full, phase, nullptr)) {
        // the copies never came: give them as long again before the block's memory goes away
        umma::mbar_wait(&full, phase, nullptr);
        set_status(p.status, GDN_ETIMEOUT);
        return;
      }
      phase ^= 1;
    }
    if (cur.hd.run && tid == 0 && cur.h == 0 && cur.ct == 0) p.rec.n[cur.hd.slot] = T;
    if (works) {
#pragma unroll
      for (int m = 0; m < RPT; ++m)
        s[m] = rst ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : *reinterpret_cast<const float4*>(st_s + (row0 + m) * CT + cq * 4);
      // ---- commit
      if (acc > 0) {
        const float2 w0 = make_float2(cW[DR_MAX], cW[DR_MAX]);
#pragma unroll
        for (int m = 0; m < RPT; ++m) {
          const float2 x = mul2(make_float2(s[m].x, s[m].y), w0);
          const float2 y = mul2(make_float2(s[m].z, s[m].w), w0);
          s[m] = make_float4(x.x, x.y, y.x, y.y);
        }
#pragma unroll 1
        for (int j = 0; j < acc; ++j) {
          const float w = cW[j];
          const float4 u = *reinterpret_cast<const float4*>(uo_s + j * CT + cq * 4);
          const float2 ua = make_float2(u.x * w, u.y * w), ub = make_float2(u.z * w, u.w * w);
          float kv[RPT];
          load_rows<RPT>(kv, rk_s + j * DK + row0);
#pragma unroll
          for (int m = 0; m < RPT; ++m) {
            const float2 kk = make_float2(kv[m], kv[m]);
            const float2 x = fma2(kk, ua, make_float2(s[m].x, s[m].y));
            const float2 y = fma2(kk, ub, make_float2(s[m].z, s[m].w));
            s[m] = make_float4(x.x, x.y, y.x, y.y);
          }
        }
      }
    }
    __syncthreads();  // the state, the old record and the sums of the tile before have been read
    if (more && warp == 0) {
      const DraftTile& w = tiles[(it + 1) & 1];
      if (w.loaded) load_tile(w, (it + 1) & 1, !w.hd.rst);
    }
    if (works && (acc > 0 || rst)) {
      float* S = p.state + (((int64_t)cur.hd.slot * p.H_v + cur.h) * DK + row0) * d_v +
                 cur.ct * CT + cq * 4;
#pragma unroll
      for (int m = 0; m < RPT; ++m) st4_stream(S + (int64_t)m * d_v, s[m]);
    }
    if (works && T > 0) {
      const int team = tid / CT, col = tid % CT;
      constexpr int QN = MAXT > TEAMS ? MAXT / TEAMS : 1;
      float qs[QN];  // q sums of tokens team, team + TEAMS, ..
#pragma unroll
      for (int g = 0; g < MAXT / G; ++g) {
        if (g * G < T) {
          const int cnt = T - g * G < G ? T - g * G : G;
          // ---- column sums S^T k_t and S^T q_t, NRW tokens at a time
#pragma unroll 1
          for (int kind = 0; kind < 2; ++kind)
#pragma unroll 1
            for (int tb = 0; tb < cnt; tb += NRW) {
              const float* vr = qk_s + (kind * T + g * G + tb) * DK + row0;
              float x[NRW][4];
#pragma unroll
              for (int v = 0; v < NRW; v += 2) {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[v][c] = x[v + 1][c] = 0.f;
                constexpr int kStep = RPT < 4 ? RPT : 4;
#pragma unroll
                for (int m = 0; m < RPT; m += kStep) {
                  float k0[kStep], k1[kStep];
                  load_rows<kStep>(k0, vr + v * DK + m);
                  load_rows<kStep>(k1, vr + (v + 1) * DK + m);
#pragma unroll
                  for (int i = 0; i < kStep; ++i) {
                    fma_row(x[v], s[m + i], k0[i]);
                    fma_row(x[v + 1], s[m + i], k1[i]);
                  }
                }
              }
              // the NRW row groups of a warp share a column quad: halve the tokens at each
              // exchange, so that a lane ends with one of them
              int mine = 0;
#pragma unroll
              for (int half = NRW / 2, step = 16; half > 0; half /= 2, step /= 2) {
                const bool hi = lane & step;
#pragma unroll
                for (int v = 0; v < half; ++v)
#pragma unroll
                  for (int c = 0; c < 4; ++c) {
                    const float keep = hi ? x[v + half][c] : x[v][c];
                    const float send = hi ? x[v][c] : x[v + half][c];
                    x[v][c] = keep + __shfl_xor_sync(0xffffffffu, send, step);
                  }
                mine += hi ? half : 0;
              }
              *reinterpret_cast<float4*>(red + ((warp * 2 + kind) * G + tb + mine) * CT + cq * 4) =
                  make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
            }
          __syncthreads();
          // ---- per column, a token per team: the right-hand side of u, the q sum
          auto col_sum = [&](int kind, int r) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) y += red[((w * 2 + kind) * G + r) * CT + col];
            return y;
          };
          const uint8_t* vs = reinterpret_cast<const uint8_t*>(cf + coef_size(D));
#pragma unroll
          for (int r0 = 0; r0 < G; r0 += TEAMS) {
            const int r = r0 + team, i = g * G + r;
            if (r < G && i < T) {
              const int at = i * CT + col;
              const float v = p.qkv_dtype == GDN_F32    ? reinterpret_cast<const float*>(vs)[at]
                              : p.qkv_dtype == GDN_BF16 ? ld(reinterpret_cast<const __nv_bfloat16*>(vs) + at)
                                                        : ld(reinterpret_cast<const __half*>(vs) + at);
              w_s[at] = cB[i] * (v - cC[i] * col_sum(0, r));
            }
          }
#pragma unroll
          for (int j = 0; j < QN; ++j) {  // the team's tokens j TEAMS + team that are in this group
            const int i = j * TEAMS + team, r = i - g * G;
            if (r >= 0 && r < G && i < T) qs[j] = col_sum(1, r);
          }
          __syncthreads();  // the sums have been read; the right-hand sides are there
        }
      }
      float u[MAXT];
#pragma unroll
      for (int i = 0; i < MAXT; ++i) u[i] = i < T ? w_s[i * CT + col] : 0.f;
      float* recu = p.rec.u + ((int64_t)cur.hd.slot * p.H_v + cur.h) * D * d_v + cur.ct * CT + col;
      const int64_t tok = (int64_t)p.H_v * d_v;
      const int64_t o0 = ((int64_t)cur.hd.c0 * p.H_v + cur.h) * d_v + cur.ct * CT + col;
      auto finish = [&](auto tt) {
        constexpr int N = decltype(tt)::value;
        // the triangular solve; rows of the tables at and behind T are zero
#pragma unroll
        for (int j = 0; j < N - 1; ++j)
#pragma unroll
          for (int i4 = (j + 1) / 4; i4 < N / 4; ++i4) {
            const float4 l = *reinterpret_cast<const float4*>(cL + j * N + 4 * i4);
            if (4 * i4 > j) u[4 * i4] = fmaf(-l.x, u[j], u[4 * i4]);
            if (4 * i4 + 1 > j) u[4 * i4 + 1] = fmaf(-l.y, u[j], u[4 * i4 + 1]);
            if (4 * i4 + 2 > j) u[4 * i4 + 2] = fmaf(-l.z, u[j], u[4 * i4 + 2]);
            u[4 * i4 + 3] = fmaf(-l.w, u[j], u[4 * i4 + 3]);
          }
#pragma unroll
        for (int r = 0; r < (N + TEAMS - 1) / TEAMS; ++r) {
          const int i = r * TEAMS + team;
          if (i < T) {
            float ui = u[r * TEAMS];
#pragma unroll
            for (int m = 1; m < TEAMS && r * TEAMS + m < N; ++m)
              ui = team == m ? u[r * TEAMS + m] : ui;
            recu[(int64_t)i * d_v] = ui;
            float o = cC[i] * qs[r];
#pragma unroll
            for (int j4 = 0; 4 * j4 < N && 4 * j4 <= r * TEAMS + TEAMS - 1; ++j4) {
              const float4 c = *reinterpret_cast<const float4*>(cP + i * N + 4 * j4);
              o = fmaf(c.x, u[4 * j4], o);
              o = fmaf(c.y, u[4 * j4 + 1], o);
              o = fmaf(c.z, u[4 * j4 + 2], o);
              o = fmaf(c.w, u[4 * j4 + 3], o);
            }
            if (p.o_dtype == GDN_F32) static_cast<float*>(p.o)[o0 + i * tok] = o;
            else st(static_cast<__nv_bfloat16*>(p.o) + o0 + i * tok, o);
          }
        }
      };
      if (TT == 4) finish(std::integral_constant<int, 4>{});
      else if (MAXT == 8 || TT == 8) finish(std::integral_constant<int, 8>{});
      else finish(std::integral_constant<int, MAXT>{});
    }
    if (!more) return;
  }
}

// The output gate of a layer draft: o = o32 / sqrt(mean(o32^2) + eps) * norm_w * SiLU(z) per
// (token, value head) row of the sequences that ran (a skipped one's rows of o stay as they
// were, and its o32 was never written). One warp per row, 8 rows per block.
template <int VPL, typename TZ, typename TO>
__global__ void __launch_bounds__(256) draft_gate_kernel(const DraftArgs p, const float* o32,
                                                         const GateArgs g) {
  const int lane = threadIdx.x & 31, n = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const DraftHeader hd = *(reinterpret_cast<const DraftHeader*>(
                               static_cast<const uint8_t*>(p.workspace) + p.ws_hdr) + n);
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (!hd.run || row >= hd.len * p.H_v) return;
  const int64_t at = (cu_at(p.cu_seqlens, n) * p.H_v + row) * p.d_v + lane * VPL;
  float o[VPL], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    o[i] = o32[at + i];
    ss = fmaf(o[i], o[i], ss);
  }
  const float inv = 1.0f / sqrtf(warp_sum(ss) / (float)p.d_v + g.eps);
  const TZ* z = static_cast<const TZ*>(g.z) + at;
  TO* out = static_cast<TO*>(g.out) + at;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    st(out + i, o[i] * inv * g.norm_w[lane * VPL + i] * silu_exact(ld(z + i)));
}

int prep_smem(int d_k, int r, int depth) {
  const int td = token_pad(depth);
  return (2 * td * (d_k + 4) + 4 * 2 * td * td + 3 * r * DR_MAX) * 4;
}
int state_smem(int d_k, int ct, int max_t, int depth, int es) {
  return (d_k * ct + depth * (d_k + ct) + 2 * late_floats(d_k, ct, depth, es) +
          2 * (st_threads(max_t) / 32) * ST_GROUP * ct + max_t * ct) * 4;
}

template <int DK, typename TX, typename TS, bool FUSED>
cudaError_t launch_prep(const DraftArgs& a, cudaStream_t s) {
  auto kern = draft_prep_kernel<DK, TX, TS, FUSED>;
  const int bytes = prep_smem(DK, a.H_v / a.H_k, a.rec.depth);
  if (bytes > 48 * 1024) {
    static std::atomic<int> smem_set[64];
    const cudaError_t e = allow_smem(kern, bytes, smem_set);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.H_k, a.n_seqs);
  cfg.blockDim = dim3(DR_THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int DK>
cudaError_t launch_prep_k(const DraftArgs& a, cudaStream_t s) {
  if (a.x) {
    const bool xb = a.x_dtype == GDN_BF16, sb = a.conv_state_dtype == GDN_BF16;
    if (xb && sb) return launch_prep<DK, __nv_bfloat16, __nv_bfloat16, true>(a, s);
    if (xb) return launch_prep<DK, __nv_bfloat16, float, true>(a, s);
    if (sb) return launch_prep<DK, float, __nv_bfloat16, true>(a, s);
    return launch_prep<DK, float, float, true>(a, s);
  }
  switch (a.qkv_dtype) {
    case GDN_F32: return launch_prep<DK, float, float, false>(a, s);
    case GDN_BF16: return launch_prep<DK, __nv_bfloat16, float, false>(a, s);
    case GDN_F16: return launch_prep<DK, __half, float, false>(a, s);
  }
  return cudaErrorInvalidValue;
}

// The state pool as [heads of all slots][d_k][d_v] fp32, a box of d_k rows x ct columns.
cudaError_t state_map(CUtensorMap* m, const DraftArgs& a, int ct) {
  const TensorMapEncodeFn enc = tensor_map_encode();
  if (!enc) return cudaErrorNotSupported;
  const int64_t heads = (int64_t)a.n_slots * a.H_v;
  if (heads > 0x7fffffff) return cudaErrorInvalidValue;
  const cuuint64_t dims[3] = {(cuuint64_t)a.d_v, (cuuint64_t)a.d_k, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)a.d_v * 4, (cuuint64_t)a.d_k * a.d_v * 4};
  const cuuint32_t box[3] = {(cuuint32_t)ct, (cuuint32_t)a.d_k, 1}, estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.state, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DK, int CT, int MAXT>
cudaError_t launch_state(const DraftArgs& a, cudaStream_t s) {
  auto kern = draft_state_kernel<DK, CT, MAXT>;
  alignas(64) CUtensorMap tm;
  cudaError_t e = state_map(&tm, a, CT);
  if (e != cudaSuccess) return e;
  const int es = a.qkv_dtype == GDN_F32 ? 4 : 2;
  const int bytes = state_smem(DK, CT, MAXT, a.rec.depth, es);
  static std::atomic<int> smem_set[64];
  // for the largest depth, so that the limit is set once
  e = allow_smem(kern, state_smem(DK, CT, MAXT, MAXT, 4), smem_set);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms == 0) return cudaErrorInvalidDevice;
  // as many blocks as fit at once: 228 KB of shared memory per SM, 1 KB of it per block reserved
  int per_sm = 228 * 1024 / (bytes + 1024 + 128);
  if (per_sm > st_blocks(MAXT)) per_sm = st_blocks(MAXT);
  const int64_t total = (int64_t)a.n_seqs * a.H_v * (a.d_v / CT);
  if (total > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(total < (int64_t)sms * per_sm ? total : (int64_t)sms * per_sm));
  cfg.blockDim = dim3(st_threads(MAXT));
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, tm);
}

template <int DK, int CT>
cudaError_t launch_state_t(const DraftArgs& a, cudaStream_t s) {
  return a.rec.depth <= 8 ? launch_state<DK, CT, 8>(a, s) : launch_state<DK, CT, DR_MAX>(a, s);
}

template <int VPL, typename TZ, typename TO>
cudaError_t launch_gate(const DraftArgs& a, const GateArgs& g, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = a.T_total < a.rec.depth ? a.T_total : a.rec.depth;  // tokens of a sequence
  cfg.gridDim = dim3((unsigned)((most * a.H_v + 7) / 8), a.n_seqs);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, draft_gate_kernel<VPL, TZ, TO>, a,
                            static_cast<const float*>(g.o), g);
}
template <int VPL>
cudaError_t launch_gate_t(const DraftArgs& a, const GateArgs& g, cudaStream_t s) {
  const bool zb = g.z_dtype == GDN_BF16, ob = g.out_dtype == GDN_BF16;
  if (zb && ob) return launch_gate<VPL, __nv_bfloat16, __nv_bfloat16>(a, g, s);
  if (zb) return launch_gate<VPL, __nv_bfloat16, float>(a, g, s);
  if (ob) return launch_gate<VPL, float, __nv_bfloat16>(a, g, s);
  return launch_gate<VPL, float, float>(a, g, s);
}

template <int DK>
cudaError_t launch_both(const DraftArgs& a0, cudaStream_t s) {
  DraftArgs a = a0;
  cudaError_t e = launch_prep_k<DK>(a, s);
  if (e != cudaSuccess) return e;
  if (a.x) {
    a.v = static_cast<uint8_t*>(a.workspace) + a.ws_v;
    a.qkv_dtype = GDN_F32;
  }
  return a.d_v % 64 == 0 ? launch_state_t<DK, 64>(a, s) : launch_state_t<DK, 32>(a, s);
}

}  // namespace

size_t draft_workspace(int H_k, int H_v, int d_k, int d_v, int64_t T_total, int n_seqs, int depth) {
  return draft_ws(H_k, H_v, d_k, d_v, T_total, n_seqs, depth).total;
}

cudaError_t launch_draft(const DraftArgs& a0, const GateArgs* gate, cudaStream_t s) {
  DraftArgs a = a0;
  const DraftWs w = draft_ws(a.H_k, a.H_v, a.d_k, a.d_v, a.T_total, a.n_seqs, a.rec.depth);
  a.pf_blocks = (int)(kStateAhead / ((int64_t)(a.H_v / a.H_k) * a.d_k * a.d_v * 4));
  a.ws_hdr = w.hdr; a.ws_qk = w.qk; a.ws_rk = w.rk; a.ws_coef = w.coef; a.ws_v = w.v;
  GateArgs g{};
  if (gate) {
    g = *gate;
    a.o = static_cast<uint8_t*>(a.workspace) + w.o32;
    a.o_dtype = GDN_F32;
    g.o = a.o;
  }
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.d_k) {
    case 32: e = launch_both<32>(a, s); break;
    case 64: e = launch_both<64>(a, s); break;
    case 128: e = launch_both<128>(a, s); break;
  }
  if (e != cudaSuccess || !gate || a.T_total == 0) return e;
  switch (a.d_v) {
    case 32: return launch_gate_t<1>(a, g, s);
    case 64: return launch_gate_t<2>(a, g, s);
    case 128: return launch_gate_t<4>(a, g, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gdn
