// attention.hip — softmax attention within documents, and its gradient.
//
//   s = scale q.k, capped by softcap tanh(s / softcap), less slope |i' - j|;
//   o = sum_j p_j v_j, p = softmax of s over the keys the token sees.
// Backward: delta = do.o, dp = do.v, ds = p (dp - delta) (1 - tanh^2),
//   dq = scale sum_j ds k_j, dk = scale sum_i ds q_i, dv = sum_i p do_i.
//
// One pass over the keys with a running maximum m and sum l: the scores never
// leave registers.  All products run on the 32x32x16 matrix instruction.  Its
// result holds one column a lane (both halves of the wavefront share 32
// columns and split the rows), so the scores are formed with the softmax's
// axis along the rows:
//   forward and dq: S^T = K Q^T: a lane is one query, its 16 registers keys;
//     row maxima and sums stay in the lane, one swap joins the two halves;
//   dk, dv: S = Q K^T: a lane is one key, its registers queries.
// The weights are then already laid out as the right operand of the next
// product (O^T = V^T P^T, dV^T = dO^T P, dK^T = Q^T dS, dQ^T = K^T dS^T) if
// its 16 contraction slots are taken in the order 8 (j / 4) + 4 half + j % 4,
// and the left operands, transposed tiles, come out of LDS through the
// transposing read (16 lanes fetch 4 rows of 16 elements and get columns):
// no lane exchange anywhere.
//
// Query heads that share a key head are packed beside each other: column
// c of a document is token c / group, head c % group, so one staged key tile
// serves all of them, and one-token requests fill the columns with heads.
#include "tokens.h"

namespace gs {

struct AttnArgs {
  Docs docs;
  int heads_q, heads_k, group, dim, causal;
  float scale, softcap;
  const float* slopes;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* o;  // backward
  const uint16_t* d;  // backward: gradient of o
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head, d_row, d_head;
  uint16_t* out0;  // forward: o; backward: dq or dk
  uint16_t* out1;  // backward: dv
  int64_t out0_row, out0_head, out1_row, out1_head;
  float* lse;    // [heads_q][rows_q]
  float* delta;  // [heads_q][rows_q]
};

constexpr int kKeys = 64;     // keys of a staged tile
constexpr int kCols = 128;    // columns of a workgroup: four wavefronts of 32
constexpr int kKeyCols = 128; // keys of a workgroup of the dk, dv kernel
constexpr int kRows = 64;     // query rows of its staged tile

template <typename T>
struct Mat;
template <>
struct Mat<Bf16> {
  typedef bf16x8 V8;
  static __device__ inline f32x16 mul(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mat<F16> {
  typedef f16x8 V8;
  static __device__ inline f32x16 mul(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// Place of 16-byte chunk c of row r in a staged tile of DT elements a row.
// Sixteen consecutive rows of one chunk (the operand read) fall on all the
// banks, and so do the eight rows by four chunks of a transposing read.
template <int DT>
__device__ inline int place(int r, int c) {
  if constexpr (DT == 128) return r * DT + ((c ^ (((r & 3) << 2) | ((r >> 2) & 3))) << 3);
  else return r * DT + ((c ^ ((((r >> 1) & 1) << 2) | ((r >> 2) & 3))) << 3);
}

// Left or right operand: rows r0 + lane % 32, contraction 16 ks + 8 half ...
template <typename T, int DT>
__device__ inline typename Mat<T>::V8 read_rows(const uint16_t* tile, int r0, int ks) {
  const int lane = threadIdx.x & 63;
  const u32x4 w = *(const u32x4*)(tile + place<DT>(r0 + (lane & 31), 2 * ks + (lane >> 5)));
  return __builtin_bit_cast(typename Mat<T>::V8, w);
}

// Left operand of the transposed tile: rows are elements d0 + lane % 32,
// contraction slots the tile's rows r0 + 8 (j / 4) + 4 half + j % 4.
template <typename T, int DT>
__device__ inline typename Mat<T>::V8 read_cols(const uint16_t* tile, int r0, int d0) {
  typedef __attribute__((address_space(3))) s16x4 L;
  const int lane = threadIdx.x & 63;
  const int r = r0 + 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int d = d0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const uint16_t* p0 = tile + place<DT>(r, d >> 3) + (d & 7);
  const uint16_t* p1 = tile + place<DT>(r + 8, d >> 3) + (d & 7);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p0);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)p1);
  const s16x8 w = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(typename Mat<T>::V8, w);
}

// Eight results of a 32-row tile (registers 8 ks ...) as the right operand's
// 16 contraction slots.
template <typename T>
__device__ inline typename Mat<T>::V8 pack_cols(const f32x16& s, int ks) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<T>(s[8 * ks + 2 * i], s[8 * ks + 2 * i + 1]);
  return __builtin_bit_cast(typename Mat<T>::V8, w);
}

// Row of result register i in a 32-row tile.
__device__ inline int result_row(int i) {
  return 8 * (i >> 2) + 4 * ((threadIdx.x & 63) >> 5) + (i & 3);
}

// x of this lane's column in both halves of the wavefront.
__device__ inline void both_halves(float x, float& lo, float& hi) {
  const uint32_t w = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  lo = __builtin_bit_cast(float, r0);
  hi = __builtin_bit_cast(float, r1);
}
__device__ inline float both_max(float x) {
  float lo, hi;
  both_halves(x, lo, hi);
  return fmaxf(lo, hi);
}
__device__ inline float both_sum(float x) {
  float lo, hi;
  both_halves(x, lo, hi);
  return lo + hi;
}

// tanh to fp32 accuracy of the result (absolute), any finite or infinite x.
__device__ inline float tanh_of(float x) {
  const float e = __builtin_amdgcn_exp2f(x * (2.0f * kLog2e));
  return 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
}

// A document as the kernels use it.
struct Doc {
  int qs, ql, ks, kl, prefix;
};
__device__ inline Doc load_doc(const Docs& d, int i) {
  Doc o;
  o.qs = clamp_start(d.q_start[i], d.rows_q);
  o.ql = clamp_len(d.q_start[i], d.q_len[i], d.rows_q);
  o.ks = clamp_start(d.k_start[i], d.rows_k);
  o.kl = clamp_len(d.k_start[i], d.k_len[i], d.rows_k);
  o.prefix = d.prefix ? min(max(d.prefix[i], 0), o.kl) : 0;
  return o;
}
// Token i sees the keys below this.
__device__ inline int key_limit(const AttnArgs& a, const Doc& d, int token) {
  return a.causal ? min(d.kl, max(token + d.kl - d.ql + 1, d.prefix)) : d.kl;
}

// 32 contiguous columns of this lane: the fragment of column c for all
// contraction steps (zeros where the column or the elements do not exist).
template <typename T, int DT>
__device__ inline void load_cols(const uint16_t* p, bool ok, int dim,
                                 typename Mat<T>::V8 (&f)[DT / 16]) {
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int ks = 0; ks < DT / 16; ++ks) {
    const int e = 16 * ks + 8 * half;
    u32x4 w = {0, 0, 0, 0};
    if (ok && e < dim) w = *(const u32x4*)(p + e);
    f[ks] = __builtin_bit_cast(typename Mat<T>::V8, w);
  }
}

// Rows [0, rows) of a key tile into LDS, zeros past `valid`.
template <int DT, int ROWS>
__device__ inline void stage_keys(uint16_t* tile, const uint16_t* base, int64_t row_stride,
                                  int valid, int dim) {
  constexpr int kChunks = DT / 8;
#pragma unroll
  for (int i = 0; i < ROWS * kChunks / 256; ++i) {
    const int x = threadIdx.x + 256 * i, r = x / kChunks, c = x % kChunks;
    u32x4 w = {0, 0, 0, 0};
    if (r < valid && c * 8 < dim) w = *(const u32x4*)(base + (int64_t)r * row_stride + c * 8);
    *(u32x4*)(tile + place<DT>(r, c)) = w;
  }
}

// Score bookkeeping shared by the three kernels: raw products of one register
// tile to scores in units of log2.  `away(i)` is |i' - j| of register i.
// With kFactor, t receives 1 - tanh^2.
template <bool kFactor, typename Away>
__device__ inline void scores(const AttnArgs& a, f32x16& s, float mul, float cap_in,
                              float cap_out, Away away, float (*t)[16]) {
  if (a.softcap > 0.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float th = tanh_of(s[i] * cap_in);
      if constexpr (kFactor) (*t)[i] = fmaf(-th, th, 1.0f);
      s[i] = th * cap_out;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] *= mul;
  }
  if (a.slopes) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] -= away(i);
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <typename T, int DT>
__global__ __launch_bounds__(256, 2) void attention_fwd_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  __shared__ __align__(16) uint16_t s_k[kKeys * DT];
  __shared__ __align__(16) uint16_t s_v[kKeys * DT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int hk = blockIdx.x % a.heads_k;
  uint32_t local, units;
  const int doc = find_document(a.docs.q_start, a.docs.q_len, a.docs.rows_q, a.docs.count,
                                a.group, kCols, blockIdx.x / a.heads_k, &local, &units);
  if (doc < 0) return;
  const Doc d = load_doc(a.docs, doc);
  // long causal rows first
  const uint32_t col0 = (units - 1 - local) * kCols;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const uint32_t c = col0 + wave * 32 + (lane & 31);
  const bool ok = c < cols;
  const int token = (int)(c / a.group), head = hk * a.group + (int)(c % a.group);
  const int lim = key_limit(a, d, token);
  const int pos = token + d.kl - d.ql;
  V8 qf[DT / 16];
  load_cols<T, DT>(a.q + (int64_t)(d.qs + token) * a.q_row + (int64_t)head * a.q_head, ok, a.dim,
                   qf);
  const float mul = a.scale * kLog2e;
  const float cap_in = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
  const float cap_out = a.softcap * kLog2e;
  const float slope = a.slopes && ok ? a.slopes[head] * kLog2e : 0.0f;

  f32x16 o[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) o[i] = (f32x16)(0.0f);
  float m = -INFINITY, l = 0.0f;
  const int last_token = (int)((min(col0 + kCols, cols) - 1) / a.group);
  const int end = key_limit(a, d, last_token);
  const int wave_lo = __builtin_amdgcn_readlane(lim, 0);
  const int wave_hi = min(__builtin_amdgcn_readlane(lim, 31), end);
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  for (int k0 = 0; k0 < end; k0 += kKeys) {
    __syncthreads();
    stage_keys<DT, kKeys>(s_k, kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
    stage_keys<DT, kKeys>(s_v, vb + (int64_t)k0 * a.v_row, a.v_row, d.kl - k0, a.dim);
    __syncthreads();
    if (k0 >= wave_hi) continue;
    f32x16 s[2];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      s[rt] = (f32x16)(0.0f);
#pragma unroll
      for (int ks = 0; ks < DT / 16; ++ks)
        s[rt] = Mat<T>::mul(read_rows<T, DT>(s_k, rt * 32, ks), qf[ks], s[rt]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const int kr = k0 + rt * 32;
      scores<false>(a, s[rt], mul, cap_in, cap_out,
                    [&](int i) { return slope * fabsf((float)(pos - kr - result_row(i))); },
                    nullptr);
      if (k0 + kKeys > wave_lo) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[rt][i] = kr + result_row(i) < lim ? s[rt][i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[rt][i]);
    }
    top = fmaxf(m, both_max(top));
    const float ref = top == -INFINITY ? 0.0f : top;
    if (__any(top > m)) {
      const float alpha = __builtin_amdgcn_exp2f(m - ref);
      l *= alpha;
#pragma unroll
      for (int i = 0; i < DT / 32; ++i) o[i] *= alpha;
      m = top;
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[rt][i] = __builtin_amdgcn_exp2f(s[rt][i] - ref);
        l += s[rt][i];
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const V8 p = pack_cols<T>(s[rt], ks);
#pragma unroll
        for (int dt = 0; dt < DT / 32; ++dt)
          o[dt] = Mat<T>::mul(read_cols<T, DT>(s_v, rt * 32 + ks * 16, dt * 32), p, o[dt]);
      }
    }
  }
  l = both_sum(l);
  if (!ok) return;
  const bool none = lim <= 0;
  const float inv = none || l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* po = a.out0 + (int64_t)(d.qs + token) * a.out0_row + (int64_t)head * a.out0_head;
#pragma unroll
  for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = dt * 32 + 8 * i + 4 * half;
      if (e < a.dim) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = none ? 0.0f : o[dt][4 * i + j] * inv;
        store_elems((T*)(po + e), x);
      }
    }
  }
  if (a.lse && half == 0)
    a.lse[(int64_t)head * a.docs.rows_q + d.qs + token] =
        none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// delta = do.o of every row and head: 16 lanes each.
template <typename T>
__global__ __launch_bounds__(256) void attention_delta_kernel(AttnArgs a) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int lane = threadIdx.x & 15;
  if (item >= (int64_t)a.docs.rows_q * a.heads_q) return;
  const int row = (int)(item / a.heads_q), head = (int)(item % a.heads_q);
  float sum = 0.0f;
  if (lane * 8 < a.dim) {
    float x[8], y[8];
    load_elems((const T*)a.o + row * a.o_row + head * a.o_head + lane * 8, x);
    load_elems((const T*)a.d + row * a.d_row + head * a.d_head + lane * 8, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 16);
  if (lane == 0) a.delta[(int64_t)head * a.docs.rows_q + row] = sum;
}

// dq: the forward's loop, with p from the stored logarithm of the sum.
template <typename T, int DT>
__global__ __launch_bounds__(256, 2) void attention_dq_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  __shared__ __align__(16) uint16_t s_k[kKeys * DT];
  __shared__ __align__(16) uint16_t s_v[kKeys * DT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int hk = blockIdx.x % a.heads_k;
  uint32_t local, units;
  const int doc = find_document(a.docs.q_start, a.docs.q_len, a.docs.rows_q, a.docs.count,
                                a.group, kCols, blockIdx.x / a.heads_k, &local, &units);
  if (doc < 0) return;
  const Doc d = load_doc(a.docs, doc);
  const uint32_t col0 = (units - 1 - local) * kCols;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const uint32_t c = col0 + wave * 32 + (lane & 31);
  const bool ok = c < cols;
  const int token = (int)(c / a.group), head = hk * a.group + (int)(c % a.group);
  const int lim = key_limit(a, d, token);
  const int pos = token + d.kl - d.ql;
  V8 qf[DT / 16], df[DT / 16];
  load_cols<T, DT>(a.q + (int64_t)(d.qs + token) * a.q_row + (int64_t)head * a.q_head, ok, a.dim,
                   qf);
  load_cols<T, DT>(a.d + (int64_t)(d.qs + token) * a.d_row + (int64_t)head * a.d_head, ok, a.dim,
                   df);
  float lse = INFINITY, delta = 0.0f;
  if (ok && lim > 0) {
    const int64_t at = (int64_t)head * a.docs.rows_q + d.qs + token;
    lse = a.lse[at] * kLog2e;
    delta = a.delta[at];
  }
  const float mul = a.scale * kLog2e;
  const float cap_in = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
  const float cap_out = a.softcap * kLog2e;
  const float slope = a.slopes && ok ? a.slopes[head] * kLog2e : 0.0f;
  f32x16 g[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) g[i] = (f32x16)(0.0f);
  const int last_token = (int)((min(col0 + kCols, cols) - 1) / a.group);
  const int end = key_limit(a, d, last_token);
  const int wave_lo = __builtin_amdgcn_readlane(lim, 0);
  const int wave_hi = min(__builtin_amdgcn_readlane(lim, 31), end);
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  for (int k0 = 0; k0 < end; k0 += kKeys) {
    __syncthreads();
    stage_keys<DT, kKeys>(s_k, kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
    stage_keys<DT, kKeys>(s_v, vb + (int64_t)k0 * a.v_row, a.v_row, d.kl - k0, a.dim);
    __syncthreads();
    if (k0 >= wave_hi) continue;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      f32x16 s = (f32x16)(0.0f), dp = (f32x16)(0.0f);
#pragma unroll
      for (int ks = 0; ks < DT / 16; ++ks) {
        s = Mat<T>::mul(read_rows<T, DT>(s_k, rt * 32, ks), qf[ks], s);
        dp = Mat<T>::mul(read_rows<T, DT>(s_v, rt * 32, ks), df[ks], dp);
      }
      const int kr = k0 + rt * 32;
      float t[16];
      scores<true>(a, s, mul, cap_in, cap_out,
                   [&](int i) { return slope * fabsf((float)(pos - kr - result_row(i))); }, &t);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[i] = __builtin_amdgcn_exp2f(s[i] - lse) * (dp[i] - delta);
      if (a.softcap > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= t[i];
      }
      if (k0 + kKeys > wave_lo) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = kr + result_row(i) < lim ? s[i] : 0.0f;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const V8 p = pack_cols<T>(s, ks);
#pragma unroll
        for (int dt = 0; dt < DT / 32; ++dt)
          g[dt] = Mat<T>::mul(read_cols<T, DT>(s_k, rt * 32 + ks * 16, dt * 32), p, g[dt]);
      }
    }
  }
  if (!ok) return;
  const bool none = lim <= 0;
  uint16_t* po = a.out0 + (int64_t)(d.qs + token) * a.out0_row + (int64_t)head * a.out0_head;
#pragma unroll
  for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = dt * 32 + 8 * i + 4 * half;
      if (e < a.dim) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = none ? 0.0f : g[dt][4 * i + j] * a.scale;
        store_elems((T*)(po + e), x);
      }
    }
  }
}

// dk and dv: a workgroup owns 128 keys of one key head and walks the tokens
// (with all their heads of the group) that may see them.
template <typename T, int DT>
__global__ __launch_bounds__(256, 2) void attention_dkv_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  __shared__ __align__(16) uint16_t s_q[kRows * DT];
  __shared__ __align__(16) uint16_t s_d[kRows * DT];
  __shared__ __align__(16) float s_lse[kRows], s_delta[kRows], s_slope[kRows];
  __shared__ __align__(16) int s_lim[kRows], s_pos[kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int hk = blockIdx.x % a.heads_k;
  uint32_t local, units;
  const int doc = find_document(a.docs.k_start, a.docs.k_len, a.docs.rows_k, a.docs.count, 1,
                                kKeyCols, blockIdx.x / a.heads_k, &local, &units);
  if (doc < 0) return;
  const Doc d = load_doc(a.docs, doc);
  const int key0 = (int)local * kKeyCols;
  const int wkey = key0 + wave * 32;
  const int key = wkey + (lane & 31);
  const bool ok = key < d.kl;
  V8 kf[DT / 16], vf[DT / 16];
  load_cols<T, DT>(a.k + (int64_t)(d.ks + key) * a.k_row + (int64_t)hk * a.k_head, ok, a.dim, kf);
  load_cols<T, DT>(a.v + (int64_t)(d.ks + key) * a.v_row + (int64_t)hk * a.v_head, ok, a.dim, vf);
  const float mul = a.scale * kLog2e;
  const float cap_in = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
  const float cap_out = a.softcap * kLog2e;
  f32x16 gk[DT / 32], gv[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) gk[i] = gv[i] = (f32x16)(0.0f);
  const uint32_t cols = (uint32_t)d.ql * a.group;
  // the first token that sees key0
  uint32_t c0 = 0;
  if (a.causal && key0 >= d.prefix)
    c0 = (uint32_t)max(key0 - (d.kl - d.ql), 0) * a.group / kRows * kRows;
  for (; c0 < cols; c0 += kRows) {
    __syncthreads();
    constexpr int kChunks = DT / 8;
#pragma unroll
    for (int i = 0; i < kRows * kChunks / 256; ++i) {
      const int x = threadIdx.x + 256 * i, r = x / kChunks, ch = x % kChunks;
      const uint32_t c = c0 + r;
      const int token = (int)(c / a.group), head = hk * a.group + (int)(c % a.group);
      u32x4 wq = {0, 0, 0, 0}, wd = {0, 0, 0, 0};
      if (c < cols && ch * 8 < a.dim) {
        wq = *(const u32x4*)(a.q + (int64_t)(d.qs + token) * a.q_row + (int64_t)head * a.q_head +
                             ch * 8);
        wd = *(const u32x4*)(a.d + (int64_t)(d.qs + token) * a.d_row + (int64_t)head * a.d_head +
                             ch * 8);
      }
      *(u32x4*)(s_q + place<DT>(r, ch)) = wq;
      *(u32x4*)(s_d + place<DT>(r, ch)) = wd;
    }
    if (threadIdx.x < kRows) {
      const uint32_t c = c0 + threadIdx.x;
      const int token = (int)(c / a.group), head = hk * a.group + (int)(c % a.group);
      const int lim = key_limit(a, d, token);
      float lse = INFINITY, delta = 0.0f, slope = 0.0f;
      if (c < cols) {
        const int64_t at = (int64_t)head * a.docs.rows_q + d.qs + token;
        if (lim > 0) {
          lse = a.lse[at] * kLog2e;
          delta = a.delta[at];
        }
        if (a.slopes) slope = a.slopes[head] * kLog2e;
      }
      s_lse[threadIdx.x] = lse;
      s_delta[threadIdx.x] = delta;
      s_slope[threadIdx.x] = slope;
      s_lim[threadIdx.x] = lim;
      s_pos[threadIdx.x] = token + d.kl - d.ql;
    }
    __syncthreads();
    if (s_lim[kRows - 1] <= wkey) continue;
    const bool full = s_lim[0] >= wkey + 32;
#pragma unroll
    for (int rt = 0; rt < kRows / 32; ++rt) {
      f32x16 s = (f32x16)(0.0f), dp = (f32x16)(0.0f);
#pragma unroll
      for (int ks = 0; ks < DT / 16; ++ks) {
        s = Mat<T>::mul(read_rows<T, DT>(s_q, rt * 32, ks), kf[ks], s);
        dp = Mat<T>::mul(read_rows<T, DT>(s_d, rt * 32, ks), vf[ks], dp);
      }
      float t[16];
      scores<true>(a, s, mul, cap_in, cap_out,
                   [&](int i) {
                     const int r = rt * 32 + result_row(i);
                     return s_slope[r] * fabsf((float)(s_pos[r] - key));
                   },
                   &t);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = rt * 32 + result_row(i);
        float p = __builtin_amdgcn_exp2f(s[i] - s_lse[r]);
        float x = p * (dp[i] - s_delta[r]);
        if (a.softcap > 0.0f) x *= t[i];
        if (!full) {
          const bool seen = key < s_lim[r];
          p = seen ? p : 0.0f;
          x = seen ? x : 0.0f;
        }
        s[i] = p;
        dp[i] = x;
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const V8 p = pack_cols<T>(s, ks), x = pack_cols<T>(dp, ks);
#pragma unroll
        for (int dt = 0; dt < DT / 32; ++dt) {
          gv[dt] = Mat<T>::mul(read_cols<T, DT>(s_d, rt * 32 + ks * 16, dt * 32), p, gv[dt]);
          gk[dt] = Mat<T>::mul(read_cols<T, DT>(s_q, rt * 32 + ks * 16, dt * 32), x, gk[dt]);
        }
      }
    }
  }
  if (!ok) return;
  uint16_t* pk = a.out0 + (int64_t)(d.ks + key) * a.out0_row + (int64_t)hk * a.out0_head;
  uint16_t* pv = a.out1 + (int64_t)(d.ks + key) * a.out1_row + (int64_t)hk * a.out1_head;
#pragma unroll
  for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = dt * 32 + 8 * i + 4 * half;
      if (e < a.dim) {
        float x[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = gk[dt][4 * i + j] * a.scale;
          y[j] = gv[dt][4 * i + j];
        }
        store_elems((T*)(pk + e), x);
        store_elems((T*)(pv + e), y);
      }
    }
  }
}

}  // namespace gs

using namespace gs;

namespace {

AttnArgs make_args(const gs_attention_config& cfg, const gs_documents& d, int64_t rows_q,
                   int64_t rows_k, const gs_heads& q, const gs_heads& k, const gs_heads& v) {
  AttnArgs a = {};
  a.docs.count = d.count;
  a.docs.rows_q = (int)rows_q;
  a.docs.rows_k = (int)rows_k;
  a.docs.q_start = d.q_start;
  a.docs.q_len = d.q_len;
  a.docs.k_start = d.k_start ? d.k_start : d.q_start;
  a.docs.k_len = d.k_len ? d.k_len : d.q_len;
  a.docs.prefix = d.prefix;
  a.heads_q = cfg.heads_q;
  a.heads_k = cfg.heads_k;
  a.group = cfg.heads_q / cfg.heads_k;
  a.dim = cfg.head_dim;
  a.causal = cfg.causal;
  a.scale = cfg.scale;
  a.softcap = cfg.softcap;
  a.slopes = cfg.slopes;
  a.q = (const uint16_t*)q.data; a.q_row = q.row; a.q_head = q.head;
  a.k = (const uint16_t*)k.data; a.k_row = k.row; a.k_head = k.head;
  a.v = (const uint16_t*)v.data; a.v_row = v.row; a.v_head = v.head;
  return a;
}

// Bound on the number of units of `step` columns (documents end inside one).
int64_t unit_bound(int64_t columns, int64_t step, int32_t count) {
  return columns / step + count;
}

template <typename T, int DT>
hipError_t run_fwd(const AttnArgs& a, hipStream_t s) {
  const int64_t units = unit_bound((int64_t)a.docs.rows_q * a.group, kCols, a.docs.count);
  attention_fwd_kernel<T, DT><<<dim3((uint32_t)(units * a.heads_k)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DT>
hipError_t run_bwd(AttnArgs a, const gs_heads& dq, const gs_heads& dk, const gs_heads& dv,
                   hipStream_t s) {
  if (a.docs.rows_q > 0) {
    const int64_t items = (int64_t)a.docs.rows_q * a.heads_q;
    attention_delta_kernel<T><<<dim3((uint32_t)((items + 15) / 16)), dim3(256), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.out0 = (uint16_t*)dq.data; a.out0_row = dq.row; a.out0_head = dq.head;
    const int64_t units = unit_bound((int64_t)a.docs.rows_q * a.group, kCols, a.docs.count);
    attention_dq_kernel<T, DT><<<dim3((uint32_t)(units * a.heads_k)), dim3(256), 0, s>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.out0 = (uint16_t*)dk.data; a.out0_row = dk.row; a.out0_head = dk.head;
  a.out1 = (uint16_t*)dv.data; a.out1_row = dv.row; a.out1_head = dv.head;
  const int64_t units = unit_bound(a.docs.rows_k, kKeyCols, a.docs.count);
  attention_dkv_kernel<T, DT><<<dim3((uint32_t)(units * a.heads_k)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

extern "C" {

size_t gs_attention_fwd_bytes(const gs_attention_config&, const gs_documents&, int64_t, int64_t) {
  return 0;
}

size_t gs_attention_bwd_bytes(const gs_attention_config& cfg, const gs_documents&, int64_t rows_q,
                              int64_t) {
  return (size_t)rows_q * cfg.heads_q * sizeof(float);
}

hipError_t gs_launch_attention_fwd(const gs_attention_config& cfg, const gs_documents& d,
                                   int64_t rows_q, int64_t rows_k, const gs_heads& q,
                                   const gs_heads& k, const gs_heads& v, const gs_heads& out,
                                   float* lse, void* workspace, hipStream_t s) {
  AttnArgs a = make_args(cfg, d, rows_q, rows_k, q, k, v);
  a.out0 = (uint16_t*)out.data; a.out0_row = out.row; a.out0_head = out.head;
  a.lse = lse;
  if (cfg.dtype == GS_BF16)
    return cfg.head_dim > 64 ? run_fwd<Bf16, 128>(a, s) : run_fwd<Bf16, 64>(a, s);
  return cfg.head_dim > 64 ? run_fwd<F16, 128>(a, s) : run_fwd<F16, 64>(a, s);
}

hipError_t gs_launch_attention_bwd(const gs_attention_config& cfg, const gs_documents& d,
                                   int64_t rows_q, int64_t rows_k, const gs_heads& q,
                                   const gs_heads& k, const gs_heads& v, const gs_heads& out,
                                   const float* lse, const gs_heads& dout, const gs_heads& dq,
                                   const gs_heads& dk, const gs_heads& dv, void* workspace,
                                   hipStream_t s) {
  AttnArgs a = make_args(cfg, d, rows_q, rows_k, q, k, v);
  a.o = (const uint16_t*)out.data; a.o_row = out.row; a.o_head = out.head;
  a.d = (const uint16_t*)dout.data; a.d_row = dout.row; a.d_head = dout.head;
  a.lse = const_cast<float*>(lse);
  a.delta = (float*)workspace;
  if (cfg.dtype == GS_BF16)
    return cfg.head_dim > 64 ? run_bwd<Bf16, 128>(a, dq, dk, dv, s)
                             : run_bwd<Bf16, 64>(a, dq, dk, dv, s);
  return cfg.head_dim > 64 ? run_bwd<F16, 128>(a, dq, dk, dv, s)
                           : run_bwd<F16, 64>(a, dq, dk, dv, s);
}

}  // extern "C"
