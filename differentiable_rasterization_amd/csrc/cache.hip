// cache.hip — keys and values brought to 8 or 4 bits as they are written into a
// cache, and read back.
//
// Each head of a token is x = low + step code, low its smallest element, step
// the (2^bits - 1)-th part of its span; codes are to nearest, formed in 64 bits.
// In 4 bits a 32-bit word holds eight elements, 2i in bits 4i and 2i + 1 in bits
// 16 + 4i: a shift and a mask then give two elements in the halves of a word.
// A quotient next to a tie of codes, which 64 bits may not tell from one, is decided
// by an exact sum.
//
// Eight elements a lane (16 bytes of a 16-bit type, 8 or 4 of codes), 8 or 16 lanes
// a head, keys and values in one launch.  20,011 tokens of 8 heads of 64, fp16 to 4
// bits: 54 MB written in 22 us, with vector instructions issued in 60% of the cycles
// (1,030 a wavefront, 300 of them 64-bit ones of the codes; places, strides and
// packing are most), and read back in 15 (3.6 TB/s; 690, of which 110 make the
// numbers).  A few tokens: a launch, 4 to 5 us.
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

// Whether code_of may take for ties in a 16-bit head what is only near them.  A quotient's
// distance from a tie is a multiple of 1 / (2 span) times the unit of the last place
// of the smallest of x, low and high, and none of 2^-36 or more is mistaken.  least:
// twice the bits of a magnitude less one, of a lane's smallest element: the whole
// wavefront acts on it, also for the lanes that do not have low or high.
template <typename T>
__device__ inline bool near_ties(uint32_t least, float span) {
  if constexpr (__is_same(T, F16)) return span > 0x1p10f;  // all are multiples of 2^-24
  // a unit is 2^-8 of the number or more; twice that for span's rounding
  return span > 0x1p26f * __builtin_bit_cast(float, least >> 1);
}
__device__ inline uint32_t twice_bits_less_one(float x) {
  return (__builtin_bit_cast(uint32_t, x) << 1) - 1;  // a zero comes last
}

// 0 where code_of(d, inv) has taken d times inv for a tie.
__device__ inline uint32_t off_tie(double d, double inv) {
  // the multiples of 2^-36 that it rounds to, in the 36 low bits
  const uint64_t w = __builtin_bit_cast(uint64_t, d * inv + 0x1.8p16);
  return (uint32_t)w | (((uint32_t)(w >> 32) ^ 8) & 15);
}

// a + b = s + e exactly (Knuth's two-sum).
__device__ inline double two_sum(double a, double b, double& e) {
  const double s = a + b, t = s - a;
  e = (a - (s - t)) + (b - t);
  return s;
}

// The code of x next to the tie of codes k and k + 1: a head's differences may have
// more bits than 64-bit numbers, so the sign of
//   2 levels (x - lo) - (2 k + 1) (hi - lo) = 2 levels x - n hi - (2 levels - n) lo,
// three exact products, is taken of their exact sum (Shewchuk's expansions).
__device__ inline int code_at_tie(float x, float lo, float hi, int levels, int k) {
  const double n = 2 * k + 1, most = 2 * levels;
  double e0, e1, e2;
  const double s0 = two_sum(most * (double)x, -n * (double)hi, e0);
  const double s1 = two_sum(-(most - n) * (double)lo, e0, e1);
  const double s2 = two_sum(s1, s0, e2);
  const double sign = s2 != 0.0 ? s2 : e2 != 0.0 ? e2 : e1;
  return sign > 0.0 ? k + 1 : sign < 0.0 ? k : k + (k & 1);
}

// A head of a token, of its keys or its values, and where it stands in the cache
// (row -1: nowhere).
struct Item {
  int64_t token, row;
  int head, kv;
  bool here;
};

// The heads of a workgroup's tokens, kLanes lanes each, kItems of them at a time
// a lane: take(items, first element, the same item by item).  Its tokens are one
// unit of a document, or where documents are no longer than one all of a document's.
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
      const auto item_of = [&](int p) {
        // what is not there repeats the last, up to what is written
        const uint32_t at = base + p * kGroups, i = min(at, items - 1);
        const int token = first + (int)(i / both), which = (int)(i % both);
        // the document's last tokens are its last keys
        const int key = token + d.kl - d.ql;
        Item o;
        o.here = at < items;
        o.token = d.qs + token;
        o.row = key < 0 ? -1 : d.ks + key;
        o.kv = which >= a.heads;
        o.head = which - (o.kv ? a.heads : 0);
        return o;
      };
      Item item[kItems];
#pragma unroll
      for (int p = 0; p < kItems; ++p) item[p] = item_of(p);
      take(item, (int)(threadIdx.x % kLanes) * 8, item_of);
    }
  }
}

// Eight elements of an item; a lane past the head's end repeats its first ones.
template <typename T>
__device__ inline void load_item(const CacheArgs& a, const Item& t, int e, float (&x)[8]) {
  load_elems((const T*)a.x[t.kv] + t.token * a.x_row[t.kv] + t.head * a.x_head[t.kv] +
                 (e < a.dim ? e : 0),
             x);
}
template <int kBits>
__device__ inline void store_item(const CacheArgs& a, const Item& t, int e, const int (&u)[8]) {
  // a token without a key is not written
  if (e < a.dim && t.here && t.row >= 0)
    store_codes<kBits>(a.codes[t.kv] + t.row * a.row[t.kv] + t.head * a.head[t.kv] + e * kBits / 8,
                       u);
}

// A head's smallest and largest element, from its lanes' eight.  One with an infinity
// or a NaN, or too wide for fp32, is wrong: it has no codes.
template <int kLanes, int kLevels>
struct Range {
  float lo, hi;
  double span, inv;
  bool wrong, none;
  __device__ inline explicit Range(const float (&x)[8]) {
    lo = hi = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      bad = bad || x[i] != x[i];
    }
    if (bad) hi = __builtin_huge_valf();
    lo = over_lanes<kLanes>(lo, [](float y, float z) { return fminf(y, z); });
    hi = over_lanes<kLanes>(hi, [](float y, float z) { return fmaxf(y, z); });
    span = (double)hi - (double)lo;
    wrong = !(span < 0x1p127);
    none = span < (double)kLeastSpan;
    inv = none || wrong ? 0.0 : (double)kLevels / span;
  }
};

template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheArgs a) {
  constexpr int kLevels = kBits == 8 ? 255 : 15;
  each_heads<kLanes>(a, [&](const Item (&item)[kItems], int e, const auto& item_of) {
    float x[kItems][8];
#pragma unroll
    for (int p = 0; p < kItems; ++p) load_item<T>(a, item[p], e, x[p]);
    bool tie = false;
    uint32_t off = 1;
#pragma unroll
    for (int p = 0; p < kItems; ++p) {
      const int kv = item[p].kv;
      const Range<kLanes, kLevels> r(x[p]);
      uint32_t least = 0xffffffffu;
      int u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = (double)x[p][i] - (double)r.lo;
        u[i] = r.wrong ? 0 : code_of(d, r.inv);
        // elements of fp32 are often small enough for near ties, which are then looked for
        if constexpr (__is_same(T, float)) off = min(off, off_tie(d, r.inv));
        else least = min(least, twice_bits_less_one(x[p][i]));
      }
      if constexpr (!__is_same(T, float)) tie = tie || near_ties<T>(least, r.hi - r.lo);
      store_item<kBits>(a, item[p], e, u);
      if (e == 0 && item[p].here && item[p].row >= 0) {
        const float nan = __builtin_nanf("");
        const int64_t at = item[p].head * a.ld[kv] + item[p].row;
        a.low[kv][at] = r.wrong ? nan : r.lo;
        a.step[kv][at] = r.wrong ? nan : r.none ? 0.0f : (float)(r.span / (double)kLevels);
      }
    }
    // Ties that may be none are rare: the wavefront's codes again, item by item, with
    // each of them decided (held beside the others it would cost a third of the
    // wavefronts, 40 us for 35).
    if (!__ballot(tie || off == 0)) return;
#pragma unroll 1
    for (int p = 0; p < kItems; ++p) {
      const Item t = item_of(p);
      float y[8];
      load_item<T>(a, t, e, y);
      const Range<kLanes, kLevels> r(y);
      int u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = (double)y[i] - (double)r.lo;
        u[i] = r.wrong ? 0 : code_of(d, r.inv);
        if (!r.wrong && off_tie(d, r.inv) == 0)
          u[i] = code_at_tie(y[i], r.lo, r.hi, kLevels, (int)(d * r.inv));
      }
      store_item<kBits>(a, t, e, u);
    }
  });
}

template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheArgs a) {
  each_heads<kLanes>(a, [&](const Item (&item)[kItems], int e, const auto&) {
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
