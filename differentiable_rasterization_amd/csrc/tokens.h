// tokens.h — what the token operators' kernels share: 16-bit and 32-bit
// element access, the look-up of a workgroup's document, and the layouts of
// the 32x32x16 matrix instruction.
#pragma once

#include "gs_common.h"

namespace gs {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLn2 = 0.6931471805599453f;

// `blocks` workgroups of `lanes` lanes, in as many launches as they need: the
// work items of one are counted in 32 bits and would wrap without an error.
// launch(first, n) starts n of them; the kernel adds `first` to its index.
template <typename F>
hipError_t launch_all(int64_t blocks, int lanes, F launch) {
  const int64_t most = ((int64_t)1 << 32) / lanes - 1;
  for (int64_t first = 0; first < blocks; first += most) {
    const int64_t n = blocks - first < most ? blocks - first : most;
    launch((uint32_t)first, dim3((uint32_t)n));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Documents as the kernels take them.  Starts and lengths come from device
// memory that the host cannot check, so every use clamps them to the rows
// the caller's buffers have.
struct Docs {
  int count;
  int rows_q, rows_k;
  const int* q_start;
  const int* q_len;
  const int* k_start;
  const int* k_len;
  const int* prefix;
};

__device__ inline int clamp_start(int start, int rows) {
  return min(max(start, 0), rows);
}
__device__ inline int clamp_len(int start, int len, int rows) {
  return min(max(len, 0), rows - clamp_start(start, rows));
}

// Inclusive sum over the wavefront's 64 lanes, by lane-to-lane moves.
__device__ inline uint32_t wave_scan(uint32_t v) {
#define GS_SCAN(ctrl, rows) \
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, true)
  GS_SCAN(0x111, 0xF);  // row_shr:1
  GS_SCAN(0x112, 0xF);  // row_shr:2
  GS_SCAN(0x114, 0xF);  // row_shr:4
  GS_SCAN(0x118, 0xF);  // row_shr:8
  GS_SCAN(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  GS_SCAN(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef GS_SCAN
  return v;
}

// A document as the kernels use it.
struct Doc {
  int qs, ql, ks, kl, prefix;
};
__device__ inline Doc load_doc(const Docs& d, int i, bool keys = true) {
  Doc o;
  const int qs = d.q_start[i], ql = d.q_len[i];
  const int ks = keys ? d.k_start[i] : qs, kl = keys ? d.k_len[i] : ql;
  const int prefix = keys && d.prefix ? d.prefix[i] : 0;
  o.qs = clamp_start(qs, d.rows_q);
  o.ql = clamp_len(qs, ql, d.rows_q);
  o.ks = clamp_start(ks, d.rows_k);
  o.kl = clamp_len(ks, kl, d.rows_k);
  o.prefix = min(max(prefix, 0), o.kl);
  return o;
}

// The document of work unit `unit`, where document d has
// ceil(n * mult / step) units, n its number of keys (kByKeys) or tokens, and
// the unit's index within it.  Every wavefront of the workgroup does the same
// scan, 64 documents at a time; all of a document's numbers are loaded
// together, since nothing else can start before they are there.  Returns -1
// past the last unit.
template <bool kByKeys>
__device__ inline int find_document(const Docs& docs, uint32_t mult, uint32_t step, uint32_t unit,
                                    uint32_t* local, uint32_t* units_of, Doc* doc,
                                    bool keys = true) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < docs.count; base += 64) {
    const int i = base + lane;
    Doc d = {0, 0, 0, 0, 0};
    if (i < docs.count) d = load_doc(docs, i, keys);
    const uint32_t n = ((uint32_t)(kByKeys ? d.kl : d.ql) * mult + step - 1) / step;
    const uint32_t cum = wave_scan(n);
    const uint64_t hit = __ballot(cum > unit);
    if (hit) {
      const int f = __ffsll((unsigned long long)hit) - 1;
      const uint32_t nf = (uint32_t)__builtin_amdgcn_readlane((int)n, f);
      *local = unit - ((uint32_t)__builtin_amdgcn_readlane((int)cum, f) - nf);
      *units_of = nf;
      doc->qs = __builtin_amdgcn_readlane(d.qs, f);
      doc->ql = __builtin_amdgcn_readlane(d.ql, f);
      doc->ks = __builtin_amdgcn_readlane(d.ks, f);
      doc->kl = __builtin_amdgcn_readlane(d.kl, f);
      doc->prefix = __builtin_amdgcn_readlane(d.prefix, f);
      return base + f;
    }
    unit -= (uint32_t)__builtin_amdgcn_readlane((int)cum, 63);
  }
  return -1;
}

// Units (ceil(len / step)) of the documents before document d, by one
// wavefront.
__device__ inline uint32_t units_before(const int* start, const int* len, int rows, int d,
                                        uint32_t step) {
  const int lane = threadIdx.x & 63;
  uint32_t n = 0;
  for (int i = lane; i < d; i += 64)
    n += ((uint32_t)clamp_len(start[i], len[i], rows) + step - 1) / step;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  return __builtin_amdgcn_readfirstlane(n);
}

// Element types.  Loads widen to fp32; stores round to nearest even, once.
struct Bf16 {
  uint16_t bits;
};
struct F16 {
  uint16_t bits;
};

__device__ inline float widen(float x) { return x; }
__device__ inline float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
__device__ inline uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ inline uint32_t pack_f16(float a, float b) {
  const f16x2 v = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// N consecutive elements (N a multiple of 2, 8- or 16-byte aligned pieces).
template <int N>
__device__ inline void load_elems(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 x = *(const f32x4*)(p + i);
      v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const f32x2 x = *(const f32x2*)(p + i);
      v[i] = x.x; v[i + 1] = x.y;
    }
  }
}
template <int N>
__device__ inline void store_elems(float* p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 x = {v[i], v[i + 1], v[i + 2], v[i + 3]};
      *(f32x4*)(p + i) = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const f32x2 x = {v[i], v[i + 1]};
      *(f32x2*)(p + i) = x;
    }
  }
}

template <typename T>
__device__ inline void unpack2(uint32_t w, float& a, float& b) {
  if constexpr (__is_same(T, Bf16)) {
    a = bf16_lo(w);
    b = bf16_hi(w);
  } else {
    const f16x2 v = __builtin_bit_cast(f16x2, w);
    a = (float)v.x;
    b = (float)v.y;
  }
}
template <typename T>
__device__ inline uint32_t pack2(float a, float b) {
  if constexpr (__is_same(T, Bf16)) return pack_bf16(a, b);
  else return pack_f16(a, b);
}

template <int W>
struct Words;
template <>
struct Words<1> { typedef uint32_t type; };
template <>
struct Words<2> { typedef u32x2 type; };
template <>
struct Words<4> { typedef u32x4 type; };

template <typename T, int N>
__device__ inline void load_elems(const T* p, float (&v)[N]) {
  typedef typename Words<N / 2>::type W;
  const W w = *(const W*)p;
  uint32_t u[N / 2];
  __builtin_memcpy(u, &w, sizeof(u));
#pragma unroll
  for (int i = 0; i < N / 2; ++i) unpack2<T>(u[i], v[2 * i], v[2 * i + 1]);
}
template <typename T, int N>
__device__ inline void store_elems(T* p, const float (&v)[N]) {
  typedef typename Words<N / 2>::type W;
  uint32_t u[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) u[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  W w;
  __builtin_memcpy(&w, u, sizeof(u));
  *(W*)p = w;
}

}  // namespace gs
