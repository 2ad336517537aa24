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
//  - draft_state_kernel, one block per (32-column tile, value head, sequence), HBM-bound: the
//    state tile in registers (loaded before the first kernel has finished), commit, column sums,
//    the T-step triangular solve per column, o and the record's u.
// The keys of a record are shared by the column tiles and value heads of a key head, so they are
// rewritten by the first kernel, which alone reads them; u belongs to one tile; the count n is
// read by the first kernel and written by the second. Nothing is read and written by different
// blocks of one kernel.
#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int DR_THREADS = 128;
constexpr int DR_TILE = 32;
constexpr int DR_MAX = 16;  // tokens per draft, at most
// per (sequence, value head) in the workspace: Lt[j][i] = beta_i D_ij (k_i.k_j) (j < i),
// P[i][j] = D_ij (q_i.k_j) (j <= i), then c, beta and the commit weights
constexpr int DR_COEF = 2 * DR_MAX * DR_MAX + 4 * DR_MAX;
constexpr int DR_L = 0, DR_P = DR_MAX * DR_MAX, DR_C = 2 * DR_MAX * DR_MAX, DR_BETA = DR_C + DR_MAX,
              DR_W = DR_BETA + DR_MAX, DR_W0 = DR_W + DR_MAX;

// What the first kernel decides about a sequence.
struct DraftHeader {
  int run;   // 0: skipped (invalid); 1: processed
  int acc;   // accepted tokens of the old record
  int len;   // new tokens
  int rst;   // starts from a zero state
};

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
      part[(warp * 2 * DR_MAX + ib + 8 * a) * DR_MAX + jb + 4 * b] = acc[a][b];
}

// TX: q, k (given) or x; TS: conv state. FUSED: from raw x.
template <int DK, typename TX, typename TS, bool FUSED>
__global__ void __launch_bounds__(DR_THREADS) draft_prep_kernel(const DraftArgs p) {
  constexpr int LDV = DK + 4, LPH = DK / 4;
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x, n = blockIdx.y;
  const int r = p.H_v / p.H_k, D = p.rec.depth;
  const bool lead = tid == 0 && hk == 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  DraftHeader* hdr = reinterpret_cast<DraftHeader*>(ws + p.ws_hdr) + n;

  // ---- validity (the same decision in every block of the sequence)
  const int64_t c0 = cu_at(p.cu_seqlens, n), c1 = cu_at(p.cu_seqlens, n + 1);
  const int slot = p.slot_ids[n];
  const bool rst = p.reset != nullptr && p.reset[n] != 0;
  const int acc = (rst || !p.accepted) ? 0 : p.accepted[n];
  int err = 0;
  if (c0 < 0 || c1 < c0 || c1 > p.T_total || c1 - c0 > D) err = GDN_EINVAL;
  else if (slot < 0 || slot >= p.n_slots) err = GDN_ESLOT;
  if (block_slot_taken(p.slot_ids, n, slot) && err == 0) err = GDN_ESLOT;
  if (err == 0 && acc != 0 && (acc < 0 || acc > D || acc > p.rec.n[slot])) err = GDN_EINVAL;
  if (err != 0) {
    if (lead) {
      set_status(p.status, err);
      *hdr = DraftHeader{0, 0, 0, 0};
    }
    return;
  }
  const int T = (int)(c1 - c0);
  if (lead) *hdr = DraftHeader{1, acc, T, rst ? 1 : 0};
  const int bs = T <= 4 ? 1 : T <= 8 ? 2 : 4, T4 = 4 * bs;

  float* vec = sm;                        // [2 DR_MAX][LDV]: k rows 0..T4-1, q rows T4..2 T4-1
  float* part = vec + 2 * DR_MAX * LDV;   // [4][2 DR_MAX][DR_MAX]
  float* ge = part + 4 * 2 * DR_MAX * DR_MAX;  // [r][DR_MAX] new decays
  float* gb = ge + r * DR_MAX;            // [r][DR_MAX] new betas
  float* go = gb + r * DR_MAX;            // [r][DR_MAX] old decays

  // ---- the accepted keys of the old record, to the workspace; the thread that reads an element
  // here is the one that overwrites it below
  float* rk = reinterpret_cast<float*>(ws + p.ws_rk) + ((int64_t)n * p.H_k + hk) * D * DK;
  float* reck = p.rec.k + ((int64_t)slot * p.H_k + hk) * D * DK;
  for (int i = tid; i < acc * LPH; i += DR_THREADS)
    reinterpret_cast<float4*>(rk)[i] = reinterpret_cast<const float4*>(reck)[i];

  // ---- gates of the key head's value heads, old and new decays
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

  // ---- q and k of the tokens into shared memory (and v to the workspace, from raw x)
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
    for (int it = 0; it < n_item; ++it) {
      int64_t ch;
      bool active;
      int jv = 0, qd = 0;
      if (warp < 2) {
        active = lane < LPH;
        ch = (int64_t)warp * p.H_k * DK + (int64_t)hk * DK + (active ? lane * 4 : 0);
      } else {
        const int item = tid - 64 + it * 64;
        active = true;
        jv = item / vq; qd = item % vq;
        const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
        ch = 2LL * p.H_k * DK + (int64_t)h * p.d_v + qd * 4;
      }
      // taps right-aligned: wa[.][3] multiplies the current token, wa[.][2 - i] the window
      float wa[4][4], win[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tap = p.d_conv - 4 + i;
          wa[j][i] = (active && tap >= 0) ? p.conv_w[(ch + j) * p.d_conv + tap] : 0.f;
        }
      // the window behind the accepted tokens: the last R rows of [conv state; recorded x[:acc]]
#pragma unroll
      for (int sl = 0; sl < 3; ++sl) {
        const int row = sl - (3 - R);  // 0 = oldest
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (active && row >= 0 && !rst) {
          const int at = row + acc;
          v = at < R ? ld4(cst + (int64_t)at * conv_dim + ch)
                     : ld4(recx + (int64_t)(at - R) * conv_dim + ch);
        }
        win[sl][0] = v.x; win[sl][1] = v.y; win[sl][2] = v.z; win[sl][3] = v.w;
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
        float4 xr[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          xr[u] = (active && tb + u < T) ? ld4(xg + (c0 + tb + u) * conv_dim + ch)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
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
          if (warp < 2) {
            const float mul = (warp == 0 ? p.q_scale : 1.0f) / sqrtf(warp_sum(ss) + p.eps);
            if (active)
              *reinterpret_cast<float4*>(vec + ((warp == 0 ? T4 : 0) + t) * LDV + lane * 4) =
                  make_float4(y[0] * mul, y[1] * mul, y[2] * mul, y[3] * mul);
          } else {
            const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
            *reinterpret_cast<float4*>(vg + ((c0 + t) * p.H_v + h) * p.d_v + qd * 4) =
                make_float4(y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
  } else {
    for (int i = tid; i < 2 * T * LPH; i += DR_THREADS) {
      const int w = i / (T * LPH), t = i / LPH - w * T, d = (i % LPH) * 4;
      const TX* src = static_cast<const TX*>(w ? p.q : p.k) + ((c0 + t) * p.H_k + hk) * DK + d;
      *reinterpret_cast<float4*>(vec + (w * T4 + t) * LDV + d) = ld4(src);
    }
  }
  __syncthreads();

  // ---- the new record's keys, and q and k for the state kernel
  float* qk = reinterpret_cast<float*>(ws + p.ws_qk) + ((int64_t)n * p.H_k + hk) * 2 * D * DK;
  for (int i = tid; i < T * LPH; i += DR_THREADS) {
    const int t = i / LPH, d = (i % LPH) * 4;
    const float4 kv = *reinterpret_cast<const float4*>(vec + t * LDV + d);
    reinterpret_cast<float4*>(reck)[i] = kv;
    reinterpret_cast<float4*>(qk)[i] = kv;
    *reinterpret_cast<float4*>(qk + (int64_t)D * DK + i * 4) =
        *reinterpret_cast<const float4*>(vec + (T4 + t) * LDV + d);
  }

  // ---- dot products (rows T..T4-1 are never read back), then the coefficient tables
  if (bs == 1) token_dots<1, DK>(vec, part);
  else if (bs == 2) token_dots<2, DK>(vec, part);
  else token_dots<4, DK>(vec, part);
  __syncthreads();
  float* coef = reinterpret_cast<float*>(ws + p.ws_coef);
  for (int i = tid; i < r * DR_MAX * DR_MAX; i += DR_THREADS) {
    const int jv = i / (DR_MAX * DR_MAX), row = (i / DR_MAX) % DR_MAX, col = i % DR_MAX;
    const int h = (p.layout & GDN_GQA_TILED) ? hk + jv * p.H_k : hk * r + jv;
    float* cf = coef + ((int64_t)n * p.H_v + h) * DR_COEF;
    if (row < T && col <= row) {
      float d = 1.f;
      for (int l = col + 1; l <= row; ++l) d *= ge[jv * DR_MAX + l];
      float kk = 0.f, qq = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        kk += part[(w * 2 * DR_MAX + row) * DR_MAX + col];
        qq += part[(w * 2 * DR_MAX + T4 + row) * DR_MAX + col];
      }
      cf[DR_P + row * DR_MAX + col] = d * qq;
      if (col < row) cf[DR_L + col * DR_MAX + row] = gb[jv * DR_MAX + row] * d * kk;
    }
    if (row == 0) {
      if (col < T) {
        float c = 1.f;
        for (int l = 0; l <= col; ++l) c *= ge[jv * DR_MAX + l];
        cf[DR_C + col] = c;
        cf[DR_BETA + col] = gb[jv * DR_MAX + col];
      }
      if (col < acc) {
        float w = 1.f;
        for (int l = col + 1; l < acc; ++l) w *= go[jv * DR_MAX + l];
        cf[DR_W + col] = w;
        if (col == 0) cf[DR_W0] = w * go[jv * DR_MAX];
      }
    }
  }
}

// TV: v; TO: o.
template <int DK, typename TV, typename TO>
__global__ void __launch_bounds__(DR_THREADS) draft_state_kernel(const DraftArgs p) {
  constexpr int RPT = DK / 16;  // state rows per thread: rg RPT .. + RPT - 1
  extern __shared__ __align__(16) float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cq = tid & 7, rg = tid >> 3;
  const int tile = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
  const int hk = khead_of(h, p.H_k, p.H_v, p.layout);
  const int d_v = p.d_v, D = p.rec.depth;
  const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);

  // ---- the state, before the first kernel's decision on this sequence is known (everything
  // read here was written before that kernel started)
  const int slot = p.slot_ids[n];
  if (slot < 0 || slot >= p.n_slots) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // this grid ends after the first one
    return;
  }
  const bool rst = p.reset != nullptr && p.reset[n] != 0;
  float* S = p.state + (((int64_t)slot * p.H_v + h) * DK + rg * RPT) * d_v + tile * DR_TILE + cq * 4;
  float4 s[RPT];
  // nothing new and nothing accepted: the state is not needed
  const bool idle = cu_at(p.cu_seqlens, n + 1) == cu_at(p.cu_seqlens, n) &&
                    (!p.accepted || p.accepted[n] == 0);
#pragma unroll
  for (int m = 0; m < RPT; ++m)
    s[m] = rst || idle ? make_float4(0.f, 0.f, 0.f, 0.f) : ld4_stream(S + (int64_t)m * d_v);
  prefetch_state_ahead<DK>(p.state, p.slot_ids, p.n_slots, p.H_v, d_v, p.pf_dist);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const DraftHeader hd = *(reinterpret_cast<const DraftHeader*>(ws + p.ws_hdr) + n);
  if (!hd.run) return;
  const int T = hd.len, acc = hd.acc;
  if (tid == 0 && h == 0 && tile == 0) p.rec.n[slot] = T;

  float* qk_s = sm;                        // [2][D][DK]
  float* rk_s = qk_s + 2 * D * DK;         // [D][DK]
  float* u_s = rk_s + D * DK;              // [D][DR_TILE]
  float* red = u_s + D * DR_TILE;          // [4 warps][2 D4][DR_TILE], D4 = D rounded up to 4
  const int D4 = (D + 3) & ~3;
  float* cf = red + 4 * 2 * D4 * DR_TILE;  // [DR_COEF]
  float* recu = p.rec.u + ((int64_t)slot * p.H_v + h) * D * d_v + tile * DR_TILE;
  {
    const float4* qk = reinterpret_cast<const float4*>(
        reinterpret_cast<const float*>(ws + p.ws_qk) + ((int64_t)n * p.H_k + hk) * 2 * D * DK);
    const float4* rk = reinterpret_cast<const float4*>(
        reinterpret_cast<const float*>(ws + p.ws_rk) + ((int64_t)n * p.H_k + hk) * D * DK);
    for (int i = tid; i < T * DK / 4; i += DR_THREADS) {
      reinterpret_cast<float4*>(qk_s)[i] = qk[i];
      reinterpret_cast<float4*>(qk_s)[D * DK / 4 + i] = qk[D * DK / 4 + i];
    }
    for (int i = tid; i < acc * DK / 4; i += DR_THREADS) reinterpret_cast<float4*>(rk_s)[i] = rk[i];
    for (int i = tid; i < acc * (DR_TILE / 4); i += DR_THREADS)
      reinterpret_cast<float4*>(u_s)[i] =
          *reinterpret_cast<const float4*>(recu + (int64_t)(i >> 3) * d_v + (i & 7) * 4);
    const float4* cg = reinterpret_cast<const float4*>(
        reinterpret_cast<const float*>(ws + p.ws_coef) + ((int64_t)n * p.H_v + h) * DR_COEF);
    for (int i = tid; i < DR_COEF / 4; i += DR_THREADS) reinterpret_cast<float4*>(cf)[i] = cg[i];
  }
  __syncthreads();

  // ---- commit
  if (acc > 0) {
    const float w0 = cf[DR_W0];
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
      s[m].x *= w0; s[m].y *= w0; s[m].z *= w0; s[m].w *= w0;
    }
    for (int j = 0; j < acc; ++j) {
      const float w = cf[DR_W + j];
      float4 u = *reinterpret_cast<const float4*>(u_s + j * DR_TILE + cq * 4);
      u.x *= w; u.y *= w; u.z *= w; u.w *= w;
      const float* kr = rk_s + j * DK + rg * RPT;
      float kv[RPT];
#pragma unroll
      for (int m = 0; m < RPT; m += 2) {
        const float2 k2 = *reinterpret_cast<const float2*>(kr + m);
        kv[m] = k2.x; kv[m + 1] = k2.y;
      }
#pragma unroll
      for (int m = 0; m < RPT; ++m) {
        s[m].x = fmaf(kv[m], u.x, s[m].x);
        s[m].y = fmaf(kv[m], u.y, s[m].y);
        s[m].z = fmaf(kv[m], u.z, s[m].z);
        s[m].w = fmaf(kv[m], u.w, s[m].w);
      }
    }
  }
  if (acc > 0 || rst) {
#pragma unroll
    for (int m = 0; m < RPT; ++m) st4_stream(S + (int64_t)m * d_v, s[m]);
  }
  if (T == 0) return;

  // ---- column sums S^T k_t and S^T q_t, four tokens at a time
  for (int tb = 0; tb < T; tb += 4) {
    float acc8[8][4];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int t = tb + (v & 3);
      const float* vr = qk_s + ((v >> 2) * D + (t < T ? t : tb)) * DK + rg * RPT;
      float kv[RPT];
#pragma unroll
      for (int m = 0; m < RPT; m += 2) {
        const float2 k2 = *reinterpret_cast<const float2*>(vr + m);
        kv[m] = k2.x; kv[m + 1] = k2.y;
      }
      float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
      for (int m = 0; m < RPT; ++m) {
        const float2 kk = make_float2(kv[m], kv[m]);
        a = fma2(make_float2(s[m].x, s[m].y), kk, a);
        b = fma2(make_float2(s[m].z, s[m].w), kk, b);
      }
      acc8[v][0] = a.x; acc8[v][1] = a.y; acc8[v][2] = b.x; acc8[v][3] = b.y;
    }
    // lanes l, l^8, l^16, l^24 share a column quad: halve the vectors at each exchange, so that
    // each lane ends with two of the eight
    const bool hi16 = lane & 16, hi8 = lane & 8;
    float a4[4][4], a2[2][4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float keep = hi16 ? acc8[v + 4][i] : acc8[v][i];
        const float send = hi16 ? acc8[v][i] : acc8[v + 4][i];
        a4[v][i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
      }
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float keep = hi8 ? a4[v + 2][i] : a4[v][i];
        const float send = hi8 ? a4[v][i] : a4[v + 2][i];
        a2[v][i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
      }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int row = (hi16 ? D4 : 0) + tb + (hi8 ? 2 : 0) + v;
      *reinterpret_cast<float4*>(red + ((warp * 2 * D4) + row) * DR_TILE + cq * 4) =
          make_float4(a2[v][0], a2[v][1], a2[v][2], a2[v][3]);
    }
  }
  __syncthreads();

  // ---- per column (lane): the triangular solve for u (every warp), o of tokens warp, warp + 4, ..
  auto col_sum = [&](int row) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) x += red[(w * 2 * D4 + row) * DR_TILE + lane];
    return x;
  };
  const int64_t c0 = cu_at(p.cu_seqlens, n);
  const TV* vg = static_cast<const TV*>(p.v) + (c0 * p.H_v + h) * d_v + tile * DR_TILE + lane;
  TO* og = static_cast<TO*>(p.o) + (c0 * p.H_v + h) * d_v + tile * DR_TILE + lane;
  const int64_t tok = (int64_t)p.H_v * d_v;
  float u[DR_MAX];
#pragma unroll
  for (int i = 0; i < DR_MAX; ++i) {
    u[i] = 0.f;
    if (i < T) u[i] = cf[DR_BETA + i] * (ld(vg + i * tok) - cf[DR_C + i] * col_sum(i));
  }
#pragma unroll
  for (int j = 0; j < DR_MAX; ++j) {
    if (j < T) {
#pragma unroll
      for (int i = j + 1; i < DR_MAX; ++i)
        if (i < T) u[i] = fmaf(-cf[DR_L + j * DR_MAX + i], u[j], u[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < DR_MAX; ++i)
    if (i < T && (i & 3) == warp) recu[(int64_t)i * d_v + lane] = u[i];
  for (int i = warp; i < T; i += 4) {
    float o = cf[DR_C + i] * col_sum(D4 + i);
#pragma unroll
    for (int j = 0; j < DR_MAX; ++j)
      if (j <= i) o = fmaf(cf[DR_P + i * DR_MAX + j], u[j], o);
    st(og + i * tok, o);
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

int prep_smem(int d_k, int r) {
  return (2 * DR_MAX * (d_k + 4) + 4 * 2 * DR_MAX * DR_MAX + 3 * r * DR_MAX) * 4;
}
int state_smem(int d_k, int depth) {
  const int d4 = (depth + 3) & ~3;
  return (3 * depth * d_k + depth * DR_TILE + 8 * d4 * DR_TILE + DR_COEF) * 4;
}

template <int DK, typename TX, typename TS, bool FUSED>
cudaError_t launch_prep(const DraftArgs& a, cudaStream_t s) {
  auto kern = draft_prep_kernel<DK, TX, TS, FUSED>;
  const int bytes = prep_smem(DK, a.H_v / a.H_k);
  if (bytes > 48 * 1024) {
    static std::atomic<int> smem_set[64];
    const cudaError_t e = allow_smem(kern, bytes, smem_set);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3(a.H_k, a.n_seqs), DR_THREADS, bytes, s>>>(a);
  return cudaGetLastError();
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

template <int DK, typename TV, typename TO>
cudaError_t launch_state(const DraftArgs& a0, cudaStream_t s) {
  auto kern = draft_state_kernel<DK, TV, TO>;
  DraftArgs a = a0;
  const int bytes = state_smem(DK, a.rec.depth);
  if (bytes > 48 * 1024) {
    static std::atomic<int> smem_set[64];
    const cudaError_t e = allow_smem(kern, bytes, smem_set);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.d_v / DR_TILE, a.H_v, a.n_seqs);
  cfg.blockDim = dim3(DR_THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int DK, typename TV>
cudaError_t launch_state_o(const DraftArgs& a, cudaStream_t s) {
  return a.o_dtype == GDN_BF16 ? launch_state<DK, TV, __nv_bfloat16>(a, s)
                               : launch_state<DK, TV, float>(a, s);
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
  switch (a.qkv_dtype) {
    case GDN_F32: return launch_state_o<DK, float>(a, s);
    case GDN_BF16: return launch_state_o<DK, __nv_bfloat16>(a, s);
    case GDN_F16: return launch_state_o<DK, __half>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t draft_workspace(int H_k, int H_v, int d_k, int d_v, int64_t T_total, int n_seqs, int depth) {
  return draft_ws(H_k, H_v, d_k, d_v, T_total, n_seqs, depth).total;
}

cudaError_t launch_draft(const DraftArgs& a0, const GateArgs* gate, cudaStream_t s) {
  DraftArgs a = a0;
  const DraftWs w = draft_ws(a.H_k, a.H_v, a.d_k, a.d_v, a.T_total, a.n_seqs, a.rec.depth);
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
