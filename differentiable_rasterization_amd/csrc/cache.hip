// cache.hip — keys and values brought to 8 or 4 bits as they are written into a
// cache, and read back.
//
// Each head of a token is x = low + step code, low its smallest element, step
// the (2^bits - 1)-th part of its span; codes are to nearest, formed in 64 bits.
// In 4 bits a 32-bit word holds eight elements, 2i in bits 4i and 2i + 1 in bits
// 16 + 4i: a shift and a mask then give two elements in the halves of a word.
//
// Eight elements a lane (16 bytes of a 16-bit type, 8 or 4 of codes), 8 or 16 lanes
// a head, keys and values in one launch.  20,011 tokens of 8 heads of 64, fp16 to 4
// bits: written in 22 us, where the codes' 64-bit arithmetic (half of about 1,000
// vector instructions a wavefront) and the reading of 41 MB weigh alike, read back in
// 15 (54 MB, 3.6 TB/s).  A few tokens: a launch, 4 to 5 us.
#include "cached.h"

namespace gs {

struct CacheArgs {
  Docs docs;
  int heads, dim;
  const void* x[2];  // keys, values
  int64_t x_row[2], x_head[2];
  uint8_t* codes[2];
  float* low[2];
  float* step[2];
  int64_t row[2], head[2], ld[2];  // strides of codes in bytes; of low and step
  int looked_up;  // units are those of the documents' tokens, else documents
  uint32_t block0;
};

constexpr int kUnit = 8;  // tokens of a workgroup

// The codes of eight elements, as they are stored.
template <int kBits>
__device__ inline void store_codes(uint8_t* p, const int (&u)[8]) {
  if constexpr (kBits == 8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)(u[4 * i] | u[4 * i + 1] << 8 | u[4 * i + 2] << 16 | u[4 * i + 3] << 24);
    *(uint32_t*)p = w[0];
    *(uint32_t*)(p + 4) = w[1];
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= (uint32_t)(u[2 * i] << 4 * i | u[2 * i + 1] << (16 + 4 * i));
    *(uint32_t*)p = w;
  }
}
template <int kBits>
__device__ inline void load_codes(const uint8_t* p, int (&u)[8]) {
  if constexpr (kBits == 8) {
    const uint32_t w[2] = {*(const uint32_t*)p, *(const uint32_t*)(p + 4)};
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (int)(w[i >> 2] >> 8 * (i & 3) & 255);
  } else {
    const uint32_t w = *(const uint32_t*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (int)(w >> (4 * (i >> 1) + 16 * (i & 1)) & 15);
  }
}

// f over groups of kLanes lanes, by lane-to-lane moves: neighbours, pairs, fours,
// eights.
template <int kCtrl>
__device__ inline float from_lane(float x) {
  const int w = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(w, w, kCtrl, 0xF, 0xF, true));
}
template <int kLanes, typename F>
__device__ inline float over_lanes(float x, F f) {
  x = f(x, from_lane<0xB1>(x));   // quad_perm 1, 0, 3, 2
  x = f(x, from_lane<0x4E>(x));   // quad_perm 2, 3, 0, 1
  x = f(x, from_lane<0x141>(x));  // row_half_mirror
  if (kLanes == 16) x = f(x, from_lane<0x140>(x));  // row_mirror
  return x;
}

// A head of a token, of its keys or its values, and where it stands in the cache
// (row -1: nowhere).
struct Item {
  int64_t token, row;
  int head, kv;
  bool here;
};

// The heads of a workgroup's tokens, kLanes lanes each, kItems of them at a time
// a lane: take(items, first element).  Its tokens are one unit of a document, or
// where documents are no longer than one all of a document's.
constexpr int kItems = 4;
template <int kLanes, typename F>
__device__ inline void each_heads(const CacheArgs& a, F take) {
  uint32_t local = 0, units;
  Doc d;
  if (!a.looked_up) d = load_doc(a.docs, (int)(a.block0 + blockIdx.x));
  else if (find_document<false>(a.docs, 1, kUnit, a.block0 + blockIdx.x, &local, &units, &d) < 0)
    return;
  const uint32_t both = 2u * (uint32_t)a.heads;
  constexpr uint32_t kGroups = 256 / kLanes;
  const int end = a.looked_up ? min((int)(local + 1) * kUnit, d.ql) : d.ql;
  for (int first = (int)local * kUnit; first < end; first += kUnit) {
    const uint32_t items = (uint32_t)min(kUnit, end - first) * both;
    for (uint32_t base = threadIdx.x / kLanes; base < items; base += kItems * kGroups) {
      Item item[kItems];
#pragma unroll
      for (int p = 0; p < kItems; ++p) {
        // what is not there repeats the last, up to what is written
        const uint32_t at = base + p * kGroups, i = min(at, items - 1);
        const int token = first + (int)(i / both), which = (int)(i % both);
        // the document's last tokens are its last keys
        const int key = token + d.kl - d.ql;
        item[p].here = at < items;
        item[p].token = d.qs + token;
        item[p].row = key < 0 ? -1 : d.ks + key;
        item[p].kv = which >= a.heads;
        item[p].head = which - (item[p].kv ? a.heads : 0);
      }
      take(item, (int)(threadIdx.x % kLanes) * 8);
    }
  }
}

template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheArgs a) {
  constexpr float kLevels = kBits == 8 ? 255.0f : 15.0f;
  each_heads<kLanes>(a, [&](const Item (&item)[kItems], int e) {
    // a lane past the head's end repeats its first elements
    const bool mine = e < a.dim;
    float x[kItems][8];
#pragma unroll
    for (int p = 0; p < kItems; ++p)
      load_elems((const T*)a.x[item[p].kv] + item[p].token * a.x_row[item[p].kv] +
                     item[p].head * a.x_head[item[p].kv] + (mine ? e : 0),
                 x[p]);
#pragma unroll
    for (int p = 0; p < kItems; ++p) {
      const int kv = item[p].kv;
      float lo = x[p][0], hi = x[p][0];
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[p][i]);
        hi = fmaxf(hi, x[p][i]);
        bad = bad || x[p][i] != x[p][i];
      }
      if (bad) hi = __builtin_huge_valf();
      lo = over_lanes<kLanes>(lo, [](float y, float z) { return fminf(y, z); });
      hi = over_lanes<kLanes>(hi, [](float y, float z) { return fmaxf(y, z); });
      // a head with an infinity or a NaN, or too wide for fp32, has no codes
      const bool wrong = !(hi - lo < 0x1p127f);
      const double span = (double)hi - (double)lo;
      const bool none = span < (double)kLeastSpan;
      const double inv = none || wrong ? 0.0 : (double)kLevels / span;
      int u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = wrong ? 0 : code_of((double)x[p][i] - (double)lo, inv);
      // a token without a key is not written
      const bool written = item[p].here && item[p].row >= 0;
      if (mine && written)
        store_codes<kBits>(
            a.codes[kv] + item[p].row * a.row[kv] + item[p].head * a.head[kv] + e * kBits / 8, u);
      if (e == 0 && written) {
        const float nan = __builtin_nanf("");
        const int64_t at = item[p].head * a.ld[kv] + item[p].row;
        a.low[kv][at] = wrong ? nan : lo;
        a.step[kv][at] = wrong ? nan : none ? 0.0f : (float)(span / (double)kLevels);
      }
    }
  });
}

template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheArgs a) {
  each_heads<kLanes>(a, [&](const Item (&item)[kItems], int e) {
    if (e >= a.dim) return;
    float lo[kItems], step[kItems];
    int u[kItems][8] = {};
#pragma unroll
    for (int p = 0; p < kItems; ++p) {
      lo[p] = step[p] = 0.0f;
      if (item[p].row < 0) continue;  // a token without a key is read as 0
      const int kv = item[p].kv;
      const int64_t at = item[p].head * a.ld[kv] + item[p].row;
      lo[p] = a.low[kv][at];
      step[p] = a.step[kv][at];
      load_codes<kBits>(
          a.codes[kv] + item[p].row * a.row[kv] + item[p].head * a.head[kv] + e * kBits / 8, u[p]);
    }
#pragma unroll
    for (int p = 0; p < kItems; ++p) {
      const int kv = item[p].kv;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lo[p] + step[p] * (float)u[p][i];
      if (item[p].here)
        store_elems((T*)a.x[kv] + item[p].token * a.x_row[kv] + item[p].head * a.x_head[kv] + e,
                    x);
    }
  });
}

namespace {

template <bool kWrite, typename T, int kBits>
hipError_t run(CacheArgs a, hipStream_t s) {
  const int64_t blocks = a.looked_up ? (int64_t)a.docs.rows_q / kUnit + a.docs.count
                                     : a.docs.count;
  return launch_all(blocks, 256, [&](uint32_t first, dim3 n) {
    a.block0 = first;
    if constexpr (kWrite) {
      if (a.dim <= 64) cache_write_kernel<T, kBits, 8><<<n, 256, 0, s>>>(a);
      else cache_write_kernel<T, kBits, 16><<<n, 256, 0, s>>>(a);
    } else {
      if (a.dim <= 64) cache_read_kernel<T, kBits, 8><<<n, 256, 0, s>>>(a);
      else cache_read_kernel<T, kBits, 16><<<n, 256, 0, s>>>(a);
    }
  });
}

template <bool kWrite>
hipError_t run(const gs_cache_config& cfg, const gs_documents& d, int64_t rows_q, int64_t rows_k,
               const gs_heads& k, const gs_heads& v, const gs_codes& kc, const gs_codes& vc,
               hipStream_t s) {
  CacheArgs a = {};
  a.docs = make_docs(d, rows_q, rows_k);
  a.looked_up = d.max_q_len == 0 || d.max_q_len > kUnit;
  a.heads = cfg.heads;
  a.dim = cfg.head_dim;
  const gs_heads* x[2] = {&k, &v};
  const gs_codes* c[2] = {&kc, &vc};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = x[i]->data; a.x_row[i] = x[i]->row; a.x_head[i] = x[i]->head;
    a.codes[i] = (uint8_t*)c[i]->codes; a.row[i] = c[i]->row; a.head[i] = c[i]->head;
    a.low[i] = c[i]->low; a.step[i] = c[i]->step; a.ld[i] = c[i]->ld;
  }
  const bool wide = kc.bits == 8;
  if (cfg.dtype == GS_F32) return wide ? run<kWrite, float, 8>(a, s) : run<kWrite, float, 4>(a, s);
  if (cfg.dtype == GS_BF16) return wide ? run<kWrite, Bf16, 8>(a, s) : run<kWrite, Bf16, 4>(a, s);
  return wide ? run<kWrite, F16, 8>(a, s) : run<kWrite, F16, 4>(a, s);
}

}  // namespace
}  // namespace gs

extern "C" {

hipError_t gs_launch_cache_write(const gs_cache_config& cfg, const gs_documents& d, int64_t rows_q,
                                 int64_t rows_k, const gs_heads& k, const gs_heads& v,
                                 const gs_codes& kc, const gs_codes& vc, hipStream_t s) {
  return gs::run<true>(cfg, d, rows_q, rows_k, k, v, kc, vc, s);
}

hipError_t gs_launch_cache_read(const gs_cache_config& cfg, const gs_documents& d, int64_t rows_q,
                                int64_t rows_k, const gs_codes& kc, const gs_codes& vc,
                                const gs_heads& k, const gs_heads& v, hipStream_t s) {
  return gs::run<false>(cfg, d, rows_q, rows_k, k, v, kc, vc, s);
}

}  // extern "C"
