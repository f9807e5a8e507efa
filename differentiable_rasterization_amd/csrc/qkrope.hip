// qkrope.hip — RMS norm of each query and key head with the rotary position
// in the same pass, and its gradient.
//
//   r = 1 / sqrt(mean x^2 + eps),  n = w x r,
//   (n_i, n_j) turned by theta = position * inv_freq_i and times amplitude,
//   pairs (i, i + R/2) or (2i, 2i + 1) for i < R/2; dims >= R keep n.
//
// Both directions move every element once and compute little: memory traffic
// is what should bound them, and does in fp32; in 16-bit types the instructions
// take as long (below).  A wavefront takes one token; 8 elements a lane
// (16 bytes of a 16-bit type), a power-of-two group of lanes a head, so the
// sum of squares is a butterfly inside the group and the other half of a
// rotated pair is either in the same lane or one shuffle away.  The angles
// depend on the token and the pair only: they are formed once a token and
// used by all its heads.  position * inv_freq is taken in 64 bits: in 32 the
// product at position 65536 would already be off by 4e-3 rad.
//
// Measured: 16,384 tokens of 20 bf16 heads of 128 elements forward, 168 MB in
// 35 us with the inputs in cache (4.8 TB/s), 39 from memory (4.3); its 21 million
// vector instructions, one a cycle and compute unit, are 35 us at 2.4 GHz too:
// bound by issue.  6,007 tokens of 24 fp32 heads of 96 forward 21 us and backward
// 31 + 4.7 for the weights (8.4 and 12.6 million instructions, 14 and 21 us;
// 277 MB in all, 67 us from memory).  Eight tokens: a kernel of 4.2 us in a call
// of 5.7 from Python.
#include "tokens.h"

namespace gs {

struct QkArgs {
  int rows, heads_q, heads_k, dim, rotary;
  int interleaved, norm;
  float eps, amplitude;
  const int* positions;
  const float* inv_freq;
  const float* wq;
  const float* wk;
  const void* q;
  const void* k;
  int64_t q_row, q_head, k_row, k_head;
  const void* dqo;  // backward: gradients of the outputs
  const void* dko;
  int64_t dqo_row, dqo_head, dko_row, dko_head;
  void* qo;  // outputs: q and k, or (backward) dq and dk
  void* ko;
  int64_t qo_row, qo_head, ko_row, ko_head;
  float* partials;  // backward: [blocks][2][dim]
  int lanes;        // lanes of a head: power of two >= dim / 8
  int items;        // wavefront items a token: 1 (all passes), or one a pass
  int passes_q, passes_k;
  uint32_t block0;  // forward: first workgroup of the launch
};

// sin and cos of t turns, t in 64 bits: reduced to the nearest quarter turn
// there, so that what is left of the angle, |x| <= pi / 4, keeps its relative
// accuracy in fp32, and so do both results near their zeros.  The series are
// Taylor's, to below 3e-8 (the cosine's next term would take its error from 1.85e-8
// to 1.77e-8, root mean square: the rest is fp32's rounding).
__device__ inline void sincos_turns(double t, float& s, float& c) {
  const double q = __builtin_rint(4.0 * t);
  const float x = (float)((t - 0.25 * q) * 6.283185307179586);
  const float y = x * x;
  float sn = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(y, sn, 8.3333333e-3f);
  sn = fmaf(y, sn, -1.6666667e-1f);
  sn = fmaf(x * y, sn, x);
  float cs = fmaf(y, 2.4801587e-5f, -1.3888889e-3f);
  cs = fmaf(y, cs, 4.1666667e-2f);
  cs = fmaf(y, cs, -0.5f);
  cs = fmaf(y, cs, 1.0f);
  const int k = (int)(q - 4.0 * __builtin_floor(0.25 * q));  // quarter 0 .. 3
  s = k & 1 ? cs : sn;
  c = k & 1 ? sn : cs;
  if (k & 2) s = -s;
  if (k == 1 || k == 2) c = -c;
}

// The lane's 8 factors: element e of chunk `chunk` turns by (c[e], s[e]), its
// partner's share signed already: y[e] = x[e] c[e] + partner[e] s[e].  With
// nothing to turn there may be no positions and no frequencies.
__device__ inline void lane_angles(const QkArgs& a, int row, int chunk, float (&c)[8],
                                   float (&s)[8]) {
  const int e0 = chunk * 8;
  const int half = a.rotary / 2;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.0f;
    s[e] = 0.0f;
  }
  if (e0 >= a.rotary) return;
  const double pos = (double)a.positions[row] * 0.15915494309189535;  // 1 / (2 pi)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int i;
    bool second;
    if (a.interleaved) {
      i = (e0 + e) >> 1;
      second = e & 1;
    } else {
      second = e0 >= half;
      i = e0 + e - (second ? half : 0);
    }
    float sn, cs;
    sincos_turns(pos * (double)a.inv_freq[i], sn, cs);
    c[e] = cs * a.amplitude;
    s[e] = (second ? sn : -sn) * a.amplitude;
  }
}

// Partner of each of the lane's elements in its rotated pair (own value for
// elements that do not turn: their factor is zero).
__device__ inline void partners(const QkArgs& a, int lane, int chunk, const float (&x)[8],
                                float (&p)[8]) {
  if (a.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
  } else {
    const int hc = a.rotary / 16;  // chunks in half the rotated part
    int src = lane;
    if (chunk < hc) src = lane + hc;
    else if (chunk < 2 * hc) src = lane - hc;
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __shfl(x[e], src, 64);
  }
}

__device__ inline float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <typename T>
__global__ __launch_bounds__(256) void qk_fwd_kernel(QkArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t item = ((int64_t)a.block0 + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int row = (int)(item / a.items);
  if (row >= a.rows) return;
  const int chunk = lane & (a.lanes - 1), sub = lane / a.lanes, per = 64 / a.lanes;
  const bool on = chunk * 8 < a.dim;
  float c[8], s[8];
  lane_angles(a, row, chunk, c, s);
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wk[e] = 1.0f;
  if (a.norm && on) {
    load_elems(a.wq + chunk * 8, wq);
    load_elems(a.wk + chunk * 8, wk);
  }
  const float inv_dim = 1.0f / (float)a.dim;
  const int passes = a.passes_q + a.passes_k;
  const int first = a.items == 1 ? 0 : (int)(item % a.items);
  const int last = a.items == 1 ? passes : first + 1;
  for (int pass = first; pass < last; ++pass) {
    const bool isq = pass < a.passes_q;
    const int head = (isq ? pass : pass - a.passes_q) * per + sub;
    const bool act = on && head < (isq ? a.heads_q : a.heads_k);
    const T* src = isq ? (const T*)a.q + row * a.q_row + head * a.q_head
                       : (const T*)a.k + row * a.k_row + head * a.k_head;
    float x[8], p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (act) load_elems(src + chunk * 8, x);
    if (a.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float r = 1.0f / sqrtf(fmaf(group_sum(ss, a.lanes), inv_dim, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (isq ? wq[e] : wk[e]);
    }
    partners(a, lane, chunk, x, p);
    if (chunk * 8 < a.rotary) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e], p[e] * s[e]);
    }
    if (act) {
      T* dst = isq ? (T*)a.qo + row * a.qo_row + head * a.qo_head
                   : (T*)a.ko + row * a.ko_row + head * a.ko_head;
      store_elems(dst + chunk * 8, x);
    }
  }
}

// Backward: dn = the transposed turn of dy, dw += dn x r,
// dx = r (g - x r^2 mean(g x)) with g = dn w.  r is formed again from x (it
// is read anyway).  A workgroup walks tokens with its grid's stride and keeps
// the weight gradients in registers; they are added over its wavefronts in
// order and left in its row of partials, which qk_weight_kernel adds in order:
// no atomics, the same bits every time.
template <typename T>
__global__ __launch_bounds__(256) void qk_bwd_kernel(QkArgs a) {
  __shared__ float s_w[4][64][9];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = lane & (a.lanes - 1), sub = lane / a.lanes, per = 64 / a.lanes;
  const bool on = chunk * 8 < a.dim;
  float wq[8], wk[8], aq[8], ak[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = wk[e] = 1.0f;
    aq[e] = ak[e] = 0.0f;
  }
  if (a.norm && on) {
    load_elems(a.wq + chunk * 8, wq);
    load_elems(a.wk + chunk * 8, wk);
  }
  const float inv_dim = 1.0f / (float)a.dim;
  const int passes = a.passes_q + a.passes_k;
  for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < a.rows; row += (int64_t)gridDim.x * 4) {
    float c[8], s[8];
    lane_angles(a, (int)row, chunk, c, s);
    for (int pass = 0; pass < passes; ++pass) {
      const bool isq = pass < a.passes_q;
      const int head = (isq ? pass : pass - a.passes_q) * per + sub;
      const bool act = on && head < (isq ? a.heads_q : a.heads_k);
      const T* px = isq ? (const T*)a.q + row * a.q_row + head * a.q_head
                        : (const T*)a.k + row * a.k_row + head * a.k_head;
      const T* pd = isq ? (const T*)a.dqo + row * a.dqo_row + head * a.dqo_head
                        : (const T*)a.dko + row * a.dko_row + head * a.dko_head;
      float x[8], d[8], p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = d[e] = 0.0f;
      if (act) {
        if (a.norm) load_elems(px + chunk * 8, x);
        load_elems(pd + chunk * 8, d);
      }
      partners(a, lane, chunk, d, p);
      if (chunk * 8 < a.rotary) {
        // the turn by -theta: the partner's share changes sign
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = fmaf(d[e], c[e], -p[e] * s[e]);
      }
      if (a.norm) {
        float ss = 0.0f, gx = 0.0f, g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = d[e] * (isq ? wq[e] : wk[e]);
          ss = fmaf(x[e], x[e], ss);
          gx = fmaf(g[e], x[e], gx);
        }
        const float r = 1.0f / sqrtf(fmaf(group_sum(ss, a.lanes), inv_dim, a.eps));
        const float m = group_sum(gx, a.lanes) * inv_dim * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // r of lanes without a head has no value where eps is 0
          const float dw = act ? d[e] * x[e] * r : 0.0f;
          if (isq) aq[e] += dw;
          else ak[e] += dw;
          d[e] = r * (g[e] - x[e] * m);
        }
      }
      if (act) {
        T* dst = isq ? (T*)a.qo + row * a.qo_row + head * a.qo_head
                     : (T*)a.ko + row * a.ko_row + head * a.ko_head;
        store_elems(dst + chunk * 8, d);
      }
    }
  }
  if (!a.norm) return;
  for (int w = 0; w < 2; ++w) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_w[wave][lane][e] = w ? ak[e] : aq[e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.dim; i += 256) {
      float sum = 0.0f;
      for (int v = 0; v < 4; ++v)
        for (int g = 0; g < per; ++g) sum += s_w[v][g * a.lanes + (i >> 3)][i & 7];
      a.partials[((int64_t)blockIdx.x * 2 + w) * a.dim + i] = sum;
    }
  }
}

// Column sums of partials [blocks][2 dim]: 16 columns a workgroup, 64 rows at
// a time, then the 64 sums in order.
__global__ __launch_bounds__(1024) void qk_weight_kernel(int blocks, int dim,
                                                         const float* __restrict__ partials,
                                                         float* dwq, float* dwk) {
  __shared__ float s_sum[64][17];
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // 2 dim is a multiple of 16
  float sum = 0.0f;
#pragma unroll 4
  for (int b = part; b < blocks; b += 64) sum += partials[(int64_t)b * 2 * dim + col];
  s_sum[part][c] = sum;
  __syncthreads();
  if (part == 0) {
#pragma unroll 8
    for (int i = 1; i < 64; ++i) sum += s_sum[i][c];
    if (col < dim) dwq[col] = sum;
    else dwk[col - dim] = sum;
  }
}

}  // namespace gs

using namespace gs;

namespace {

int next_pow2(int n) {
  int p = 1;
  while (p < n) p <<= 1;
  return p;
}

QkArgs make_args(const gs_qk_config& cfg, int64_t rows, const int32_t* positions,
                 const float* inv_freq, const float* wq, const float* wk, const gs_heads& q,
                 const gs_heads& k, const gs_heads& qo, const gs_heads& ko) {
  QkArgs a = {};
  a.rows = (int)rows;
  a.heads_q = cfg.heads_q;
  a.heads_k = cfg.heads_k;
  a.dim = cfg.head_dim;
  a.rotary = cfg.rotary_dim;
  a.interleaved = cfg.interleaved;
  a.norm = cfg.norm;
  a.eps = cfg.eps;
  a.amplitude = cfg.amplitude;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.wq = wq;
  a.wk = wk;
  a.q = q.data; a.q_row = q.row; a.q_head = q.head;
  a.k = k.data; a.k_row = k.row; a.k_head = k.head;
  a.qo = qo.data; a.qo_row = qo.row; a.qo_head = qo.head;
  a.ko = ko.data; a.ko_row = ko.row; a.ko_head = ko.head;
  a.lanes = next_pow2((cfg.head_dim + 7) / 8);
  const int per = 64 / a.lanes;
  a.passes_q = (cfg.heads_q + per - 1) / per;
  a.passes_k = (cfg.heads_k + per - 1) / per;
  return a;
}

// Workgroups of the backward: enough to fill the chip several times over, few
// enough that their partial weight gradients stay a small sum.
int bwd_blocks(int64_t rows) {
  const int64_t b = (rows + 3) / 4;
  return (int)(b < 1024 ? b : 1024);
}

}  // namespace

extern "C" {

size_t gs_qk_bwd_workspace_bytes(const gs_qk_config& cfg, int64_t rows) {
  return cfg.norm ? (size_t)bwd_blocks(rows) * 2 * cfg.head_dim * sizeof(float) : 0;
}

hipError_t gs_launch_qk_fwd(const gs_qk_config& cfg, int64_t rows, const int32_t* positions,
                            const float* inv_freq, const float* wq, const float* wk,
                            const gs_heads& q, const gs_heads& k, const gs_heads& qo,
                            const gs_heads& ko, hipStream_t s) {
  QkArgs a = make_args(cfg, rows, positions, inv_freq, wq, wk, q, k, qo, ko);
  const int passes = a.passes_q + a.passes_k;
  // a wavefront a token amortises the angles; with too few tokens to fill the
  // chip, a wavefront a pass
  a.items = rows * passes <= 4096 ? passes : 1;
  const int64_t blocks = (rows * a.items + 3) / 4;
  const dim3 block(256);
  return launch_all(blocks, 256, [&](uint32_t first, dim3 grid) {
    a.block0 = first;
    if (cfg.dtype == GS_F32) qk_fwd_kernel<float><<<grid, block, 0, s>>>(a);
    else if (cfg.dtype == GS_BF16) qk_fwd_kernel<Bf16><<<grid, block, 0, s>>>(a);
    else qk_fwd_kernel<F16><<<grid, block, 0, s>>>(a);
  });
}

hipError_t gs_launch_qk_bwd(const gs_qk_config& cfg, int64_t rows, const int32_t* positions,
                            const float* inv_freq, const float* wq, const float* wk,
                            const gs_heads& q, const gs_heads& k, const gs_heads& dqo,
                            const gs_heads& dko, const gs_heads& dq, const gs_heads& dk,
                            float* dwq, float* dwk, void* workspace, hipStream_t s) {
  QkArgs a = make_args(cfg, rows, positions, inv_freq, wq, wk, q, k, dq, dk);
  a.dqo = dqo.data; a.dqo_row = dqo.row; a.dqo_head = dqo.head;
  a.dko = dko.data; a.dko_row = dko.row; a.dko_head = dko.head;
  a.partials = (float*)workspace;
  const int blocks = bwd_blocks(rows);  // 0 rows: only the (zero) weight gradients
  if (blocks > 0) {
    const dim3 grid(blocks), block(256);
    if (cfg.dtype == GS_F32) qk_bwd_kernel<float><<<grid, block, 0, s>>>(a);
    else if (cfg.dtype == GS_BF16) qk_bwd_kernel<Bf16><<<grid, block, 0, s>>>(a);
    else qk_bwd_kernel<F16><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !cfg.norm) return e;
  }
  qk_weight_kernel<<<dim3(2 * cfg.head_dim / 16), dim3(1024), 0, s>>>(
      blocks, cfg.head_dim, (const float*)workspace, dwq, dwk);
  return hipGetLastError();
}

}  // extern "C"
