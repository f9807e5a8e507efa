// cached.hip — attention of a few new tokens over a cache of 8- or 4-bit codes,
// with keys that many requests share read once for all of them.
//
//   key j = low_j + step_j u_j:  q.k_j = step_j (q.u_j) + low_j sum(q),
//   sum_j p_j v_j = sum_j (p_j step_j) (u_j - mid) + sum_j p_j (low_j + mid step_j).
// Codes are whole numbers that the 16-bit types hold exactly, so both products
// run on the matrix unit from codes brought to 16 bits in registers; only the
// weights p_j step_j are rounded, to fp16 (11 bits) for either type: taken
// relative to a power of two near the column's largest, so that they stay in its
// range.  Codes are centred there, since the rounding of a weight acts on the
// whole of what it multiplies.
//
// Query heads that share a key head stand beside each other: column c of a
// document is token c / group, head c % group.  A wavefront takes 32 keys at a
// time by 16 or 32 columns, on the 16x16x32 instruction:
//   S^T = K Q^T: lane l has column l % 16 and keys 4 (l / 16) + 0..3 of both
//     16-key halves; its 8 weights are the right operand of
//   O^T = V^T P^T, if the contraction runs over the keys in that order; the left
//     operand takes single elements of those keys' rows, which each lane loads
//     itself (16 lanes a row) and pairs by byte permutes.
// So scores and weights never leave their registers; what a key's low and step make
// of a score or a weight passes through LDS, 512 bytes a tile, and where there are
// many columns so do the operands, for all four wavefronts.
//
// Keys are cut into pieces where there are few columns; a second kernel joins a
// token's pieces and those of the keys it shares.
//
// What bounds it.  One token a request: reading the codes (four caches of 120,001
// keys in all, 4 heads of 128 in 8 bits: 131 MB in 37.6 us, 3.5 TB/s, and 5 for the
// join; a large sum that only reads has 3.9).  Many columns: vector instructions and
// matrix products of two wavefronts a SIMD that overlap little (1,024 tokens over
// 32,768 keys, 16 heads of 128 over 4: 416 us, 0.65 PFLOP/s, up to 20% more in the
// first 50 calls after a pause; vector issue in 52% of the cycles, matrix unit at work
// in 26).  Small calls: two launches and a chain of dependent loads (document, codes,
// pieces), about 15 us.
#include "cached.h"

namespace gs {

typedef _Float16 f16x2v __attribute__((ext_vector_type(2)));

struct CachedArgs {
  Docs docs;    // of this pass
  Docs shared;  // join: count 0 without shared keys
  int heads_q, heads_k, group, dim, causal;
  float scale, softcap;
  const float* slopes;
  const uint16_t* q;
  int64_t q_row, q_head;
  const uint8_t *kc, *vc;  // codes; strides in bytes
  int64_t kc_row, kc_head, vc_row, vc_head;
  const float *klow, *kstep, *vlow, *vstep;  // [heads_k][ld]
  int64_t k_ld, v_ld;
  uint16_t* out;
  int64_t out_row, out_head;
  float* lse;
  float* part_ml;  // [pieces][heads_q][rows_q][2]
  float* part_o;   // [pieces][heads_q][rows_q][dim]
  int pieces, pieces_shared;  // at most, of a document
  int piece, piece_shared;    // keys of one
  int first_piece;  // of this pass, in the arrays above
  int whole;        // one piece and nothing shared: the result is written at once
  int looked_up;    // column tiles are units of the grid, else documents
  int width;        // columns of a workgroup
  uint32_t units, blocks, block0;
};

constexpr int kStepKeys = 128;  // keys the four wavefronts take at a time

// Keys of a piece of a document of kl keys.  Pieces have one size in all
// documents, so that long ones do not end late; one that is longer than the
// caller said gets larger pieces.
__device__ inline int piece_keys(int kl, int pieces, int piece) {
  const int n = (int)(((int64_t)kl + pieces - 1) / pieces);
  return max((n + kStepKeys - 1) / kStepKeys * kStepKeys, piece);
}

// Token i sees the keys below this.
__device__ inline int key_limit(const CachedArgs& a, const Doc& d, int token) {
  return a.causal ? min(d.kl, max(token + d.kl - d.ql + 1, d.prefix)) : d.kl;
}

// x of lane l % 16 in all four rows of 16 lanes: largest, sum.
template <typename F>
__device__ inline float across(float x, F f) {
  uint32_t w = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const uint32_t a0 = a[0], a1 = a[1];
  const float y = f(__builtin_bit_cast(float, a0), __builtin_bit_cast(float, a1));
  w = __builtin_bit_cast(uint32_t, y);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t b0 = b[0], b1 = b[1];
  return f(__builtin_bit_cast(float, b0), __builtin_bit_cast(float, b1));
}
__device__ inline float across_max(float x) {
  return across(x, [](float p, float q) { return fmaxf(p, q); });
}
__device__ inline float across_sum(float x) {
  return across(x, [](float p, float q) { return p + q; });
}

template <typename T>
struct Mat16;
template <>
struct Mat16<Bf16> {
  typedef bf16x8 V8;
  static __device__ inline f32x4 mul(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mat16<F16> {
  typedef f16x8 V8;
  static __device__ inline f32x4 mul(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// (lo, hi) fp16 numbers of a word, times mul, plus add: exact here.
__device__ inline uint32_t fma_f16(uint32_t w, _Float16 mul, _Float16 add) {
  const f16x2v m = {mul, mul}, c = {add, add};
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_fma(__builtin_bit_cast(f16x2v, w), m, c));
}

// Eight codes as key operand, x = (code - kOff) / kMul exactly.
template <typename T, int kBits>
struct KeyCodes {
  // 8 bits in bf16: the code itself; in fp16: (u - 128) / 512.
  // 4 bits: 1 + u / 16, made by placing the four bits in a mantissa.
  static constexpr float kMul = kBits == 4 ? 16.0f : __is_same(T, Bf16) ? 1.0f : 512.0f;
  static constexpr float kOff = kBits == 4 ? -16.0f : __is_same(T, Bf16) ? 0.0f : 128.0f;
  static __device__ inline typename Mat16<T>::V8 operand(const uint32_t* w) {
    uint32_t o[4];
    if constexpr (kBits == 4) {
      constexpr bool kB = __is_same(T, Bf16);
      constexpr uint32_t one = kB ? 0x3f803f80u : 0x3c003c00u;
      constexpr uint32_t mask = kB ? 0x00780078u : 0x03c003c0u;
      constexpr int place = kB ? 3 : 6;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int right = 4 * i - place;
        o[i] = ((right >= 0 ? w[0] >> (right & 31) : w[0] << (-right & 31)) & mask) | one;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i >> 1], at = 16 * (i & 1);
        if constexpr (__is_same(T, Bf16)) {
          o[i] = pack_bf16((float)(x >> at & 255), (float)(x >> (at + 8) & 255));
        } else {
          // two bytes as the subnormal numbers u 2^-24
          const uint32_t pair = __builtin_amdgcn_perm(0, x, i & 1 ? 0x0c030c02u : 0x0c010c00u);
          o[i] = fma_f16(pair, (_Float16)32768.0f, (_Float16)-0.25f);
        }
      }
    }
    return __builtin_bit_cast(typename Mat16<T>::V8, u32x4{o[0], o[1], o[2], o[3]});
  }
};

// What a lane loads of the eight rows of values it has, and element e of all of
// them as operand: (code - kMid) / 512.
template <int kBits, int DT>
struct ValueCodes {
  static constexpr int kElems = DT / 16;  // of a row, a lane
  static constexpr int kWords = kBits == 8 ? kElems / 4 : 1;
  static constexpr float kMid = kBits == 8 ? 128.0f : 8.0f;
  // First byte of lane n's part of a row (4 bits, 64 elements: half a word, of
  // the even or the odd elements), and its first element.
  static __device__ inline int byte_of(int n) { return n * kElems * kBits / 8; }
  static __device__ inline int first_of(int n) {
    return kBits == 4 && DT == 64 ? 8 * (n >> 1) : n * kElems;
  }
  // Element e of lane n's part.
  static __device__ inline int element(int n, int e) {
    if (kBits == 8) return n * kElems + e;
    if (DT == 64) return 8 * (n >> 1) + 2 * e + (n & 1);
    return 8 * n + (e < 4 ? 2 * e : 2 * (e - 4) + 1);
  }
  static __device__ inline f16x8 operand(const uint32_t (&v)[8][kWords], int e) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBits == 8) {
        const uint32_t c = e & 3;
        const uint32_t pair = __builtin_amdgcn_perm(v[2 * i + 1][e >> 2], v[2 * i][e >> 2],
                                                    0x0c000c00u | c | (4 + c) << 16);
        o[i] = fma_f16(pair, (_Float16)32768.0f, (_Float16)-0.25f);
      } else {
        const uint32_t p = __builtin_amdgcn_perm(v[2 * i + 1][0], v[2 * i][0],
                                                 e < 4 ? 0x05040100u : 0x07060302u) >>
                           (e & 2 ? 8 : 0);
        o[i] = e & 1 ? fma_f16(p & 0x00f000f0u, (_Float16)2048.0f, (_Float16)-0.015625f)
                     : fma_f16(p & 0x000f000fu, (_Float16)32768.0f, (_Float16)-0.015625f);
      }
    }
    return __builtin_bit_cast(f16x8, u32x4{o[0], o[1], o[2], o[3]});
  }
};

// Numbers of a wavefront's 32 keys in LDS: what scores are multiplied by and what is
// added, the same of weights.
constexpr int kNumbers = 4 * 32;

// The codes of 32 keys as a lane has them.  Rows of the cache are reached through
// a buffer descriptor that ends with the last of `valid` rows: codes of keys past
// that, and of elements past dim, whose offset is past every end, are zero.
template <int kBits, int DT>
struct KeyRows {
  static constexpr int kPieces = DT / 64;        // of 16 elements, of a key, a lane
  static constexpr int kPieceWords = kBits / 2;  // of such a piece
  uint32_t w[2][kPieces * kPieceWords];
  uint32_t at[kPieces];  // of this lane's first key
  __device__ inline void start(int row, int dim) {
    const int n = threadIdx.x & 15, kg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = kg * (DT / 4) + 16 * i;
      at[i] = e < dim ? (uint32_t)(n * row + e * kBits / 8) : 0x80000000u;
      // not to be taken for one of two constants, with a branch for each
      asm("" : "+v"(at[i]));
    }
  }
  __device__ inline void load(const uint8_t* base, int row, int bytes) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes,
                                                        0x00027000);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int from = (int)(at[i] + (uint32_t)(16 * t * row));
        uint32_t* to = w[t] + i * kPieceWords;
        if constexpr (kBits == 8) {
          const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rsrc, from, 0, 0);
          to[0] = x.x; to[1] = x.y; to[2] = x.z; to[3] = x.w;
        } else {
          const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, from, 0, 0);
          to[0] = x.x; to[1] = x.y;
        }
      }
  }
};
template <int kBits, int DT>
struct ValueRows {
  typedef ValueCodes<kBits, DT> V;
  uint32_t w[8][V::kWords];
  uint32_t at;  // of this lane's first key
  __device__ inline void start(int row, int dim) {
    const int n = threadIdx.x & 15, kg = (threadIdx.x & 63) >> 4;
    at = V::first_of(n) < dim ? (uint32_t)(4 * kg * row + V::byte_of(n)) : 0x80000000u;
    asm("" : "+v"(at));
  }
  __device__ inline void load(const uint8_t* base, int row, int bytes) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, bytes,
                                                        0x00027000);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int from = (int)(at + (uint32_t)((16 * (j >> 2) + (j & 3)) * row));
      if constexpr (V::kWords == 2) {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rsrc, from, 0, 0);
        w[j][0] = x.x; w[j][1] = x.y;
      } else if constexpr (kBits == 4 && DT == 64) {
        w[j][0] = __builtin_amdgcn_raw_buffer_load_b16(rsrc, from, 0, 0);
      } else {
        w[j][0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, from, 0, 0);
      }
    }
  }
};

// Weights are 2^(score - reference): up to 1 when the reference is taken, and it
// moves only when a score has passed it by kGrowth, so they stay below 2^6.  Sums of
// weights times values then end where those of the values alone reach 2^122.
constexpr float kGrowth = 6.0f;

// Weights times steps become fp16 numbers relative to a unit, a power of two: the
// largest lies in [2^kUnitRoom, 2 2^kUnitRoom) when the unit is taken, and the unit
// moves when one passes 2^15.  What is below 2^-22 of a token's largest loses bits.
constexpr int kUnitRoom = 8;
constexpr float kMostWeight = 0x1p15f;

__device__ inline int exponent_of(float x) {  // with its bias of 127; x >= 0
  return (int)(__builtin_bit_cast(uint32_t, x) >> 23);
}
__device__ inline float power_of(int e) { return __builtin_bit_cast(float, (uint32_t)e << 23); }

// kMode: plain scores, capped ones, or a distance bias (with or without a cap).
constexpr int kPlain = 0, kCapped = 1, kBiased = 2;

// What a workgroup takes: the piece of a document's keys, of one head, and the
// columns from first to end.  All heads of the same keys go to one XCD, one after
// the other: rows of neighbouring heads share lines.
struct Work {
  Doc d;
  int hk, piece, key0, keys;
  int first, end, cols;
};
__device__ inline bool find_work(const CachedArgs& a, uint32_t block, int width, Work& w) {
  const uint32_t turn = block >> 3;
  w.hk = (int)(turn % (uint32_t)a.heads_k);
  const uint32_t place = turn / (uint32_t)a.heads_k * 8 + (block & 7);
  const uint32_t unit = place % a.units;
  w.piece = (int)(place / a.units);
  if (w.piece >= a.pieces) return false;
  w.first = 0;
  w.end = 0x7fffffff;
  if (a.looked_up) {
    uint32_t local, units;
    if (find_document<false>(a.docs, (uint32_t)a.group, (uint32_t)width, unit, &local, &units,
                             &w.d) < 0)
      return false;
    w.first = (int)local * width;
    w.end = w.first + width;
  } else {
    w.d = load_doc(a.docs, (int)unit);
  }
  w.cols = w.d.ql * a.group;
  w.end = min(w.end, w.cols);
  w.keys = piece_keys(w.d.kl, a.pieces, a.piece);
  if (w.piece > 0 && (int64_t)w.piece * w.keys >= w.d.kl) return false;
  w.key0 = w.piece * w.keys;
  return true;
}

// A wavefront's tiles of 32 keys on their way from memory: its lanes' codes, and
// of one key low and step (lanes 0..31 have the keys' own, lanes 32..63 their
// values'), which that lane brings to what a score or a weight needs of it, for
// all that use it, through LDS.
template <typename T, int kBits, int DT>
struct Tiles {
  typedef KeyCodes<T, kBits> K;
  typedef ValueCodes<kBits, DT> V;
  KeyRows<kBits, DT> k;
  ValueRows<kBits, DT> v;
  float low, step;
  const uint8_t *kp, *vp;  // of the next tile
  const float *lows, *steps;
  int k_row, v_row, head_bytes, kl, key_end;

  __device__ inline void start(const CachedArgs& a, const Work& w, int key, int end) {
    const bool of_values = (threadIdx.x & 32) != 0;
    k_row = (int)a.kc_row;
    v_row = (int)a.vc_row;
    head_bytes = a.dim * kBits / 8;
    kl = w.d.kl;
    key_end = end;
    kp = a.kc + (int64_t)(w.d.ks + key) * a.kc_row + w.hk * a.kc_head;
    vp = a.vc + (int64_t)(w.d.ks + key) * a.vc_row + w.hk * a.vc_head;
    const int64_t at = of_values ? w.hk * a.v_ld + w.d.ks : w.hk * a.k_ld + w.d.ks;
    lows = (of_values ? a.vlow : a.klow) + at;
    steps = (of_values ? a.vstep : a.kstep) + at;
    k.start(k_row, a.dim);
    v.start(v_row, a.dim);
    low = step = 0.0f;
    load_numbers(key);
    k.load(kp, k_row, bytes(key, k_row));
    v.load(vp, v_row, bytes(key, v_row));
  }
  // From a tile's first key to its last one's end; none past the end.
  __device__ inline int bytes(int key, int row) const {
    return key < key_end ? (min(32, kl - key) - 1) * row + head_bytes : 0;
  }
  __device__ inline void load_numbers(int key) {
    if (key >= key_end) return;
    const int at = key + min((int)(threadIdx.x & 31), kl - key - 1);
    low = lows[at];
    step = steps[at];
  }
  __device__ inline void next_keys(int key) {
    kp += (int64_t)kStepKeys * k_row;
    k.load(kp, k_row, bytes(key, k_row));
  }
  __device__ inline void next_values(int key) {
    vp += (int64_t)kStepKeys * v_row;
    v.load(vp, v_row, bytes(key, v_row));
  }
  __device__ inline void leave_numbers(float* nums, float to_log2) const {
    const int lane = threadIdx.x & 63;
    const bool of_values = lane >= 32;
    nums[2 * (lane & 32) + (lane & 31)] = of_values ? step : step * (K::kMul * to_log2);
    nums[2 * (lane & 32) + 32 + (lane & 31)] =
        fmaf(step, of_values ? V::kMid : K::kOff, low) * (of_values ? 1.0f : to_log2);
  }
};

// CT times 16 columns of a wavefront: queries, and the running sums of a softmax.
// Weights are relative to ref, which a score above most moves; weights times steps
// are fp16 numbers times 1 / per_unit, a power of two.  Both belong to the column and
// move by what it sees alone, by powers of two: keys that it does not see, and what
// stands in the columns beside it, leave its bits as they are.
template <typename T, int kBits, int DT, int CT, int kMode>
struct Columns {
  typedef ValueCodes<kBits, DT> V;
  typedef typename Mat16<T>::V8 V8;
  static constexpr int kSteps = DT / 32;    // of the scores' contraction
  static constexpr int kElems = V::kElems;  // products of 16 elements of the values
  V8 q[CT][kSteps];
  float qsum[CT], slope[CT];
  int limit[CT], pos[CT];
  f32x4 o[CT][kElems];
  float ref[CT], most[CT], l[CT], mean[CT], per_unit[CT];

  // Columns past the last one repeat it, and are not stored.
  __device__ inline void start(const CachedArgs& a, const Work& w, int col0) {
    const int n = threadIdx.x & 15, kg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int c = min(col0 + 16 * ct + n, w.cols - 1);
      const int token = c / a.group, head = w.hk * a.group + c % a.group;
      const uint16_t* p = a.q + (int64_t)(w.d.qs + token) * a.q_row + head * a.q_head;
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int e = kg * (DT / 4) + 8 * s;
        u32x4 x = {0, 0, 0, 0};
        if (e < a.dim) x = *(const u32x4*)(p + e);
        q[ct][s] = __builtin_bit_cast(V8, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y, z;
          unpack2<T>(x[i], y, z);
          sum += y + z;
        }
      }
      qsum[ct] = across_sum(sum);
      limit[ct] = key_limit(a, w.d, token);
      pos[ct] = token + w.d.kl - w.d.ql;
      slope[ct] = kMode == kBiased ? a.slopes[head] * kLog2e : 0.0f;
      most[ct] = -INFINITY;
      ref[ct] = l[ct] = mean[ct] = 0.0f;
      per_unit[ct] = 0x1p126f;
#pragma unroll
      for (int e = 0; e < kElems; ++e) o[ct][e] = (f32x4)(0.0f);
    }
  }

  __device__ inline void scale_sums(int ct, int by) {
#pragma unroll
    for (int e = 0; e < kElems; ++e)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[ct][e][r] = __builtin_amdgcn_ldexpf(o[ct][e][r], by);
  }
  // The weights so far are 2^-n of what they were: so is the unit, down to 2^-126.
  __device__ inline void shrink(int ct, int n) {
    const int e = exponent_of(per_unit[ct]), now = min(e + n, 253);
    per_unit[ct] = power_of(now);
    if (__ballot(now < e + n)) scale_sums(ct, now - e - n);
  }
  // Room for a weight times step of this size, over the column's lanes.
  __device__ inline void make_room(int ct, float size) {
    const float top = across_max(size);
    const int e = exponent_of(per_unit[ct]);
    const bool grows = top * per_unit[ct] > kMostWeight && top < __builtin_huge_valf();
    const int now = grows ? 2 * 127 + kUnitRoom - exponent_of(top) : e;
    per_unit[ct] = power_of(now);
    scale_sums(ct, now - e);
  }
  __device__ inline float unit(int ct) const { return power_of(254 - exponent_of(per_unit[ct])); }

  __device__ inline f32x4 step_of(const float* nums, int t, int kg) const {
    return *(const f32x4*)(nums + 64 + 16 * t + 4 * kg);
  }
  __device__ inline f32x4 mean_of(const float* nums, int t, int kg) const {
    return *(const f32x4*)(nums + 96 + 16 * t + 4 * kg);
  }

  // Weights of 32 keys from their scores' products s.  first: this lane's keys are
  // first + 0..3 and first + 16 + 0..3.
  __device__ inline void weigh(const CachedArgs& a, const float* nums, const f32x4 (&s)[2][CT],
                               bool masked, int first, int key_end, f16x8 (&w)[CT]) {
    const int kg = (threadIdx.x & 63) >> 4;
    const float cap = a.softcap * kLog2e;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float y[8], top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const f32x4 kmul = *(const f32x4*)(nums + 16 * t + 4 * kg);
        const f32x4 kadd = *(const f32x4*)(nums + 32 + 16 * t + 4 * kg);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float& z = y[4 * t + r];
          if constexpr (kMode == kPlain)
            z = fmaf(s[t][ct][r], kmul[r], fmaf(kadd[r], qsum[ct], -ref[ct]));
          else
            z = fmaf(s[t][ct][r], kmul[r], kadd[r] * qsum[ct]);
        }
      }
      if constexpr (kMode != kPlain) {
        if (a.softcap > kWideCap) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fmaf(cap, tanh_wide(y[j]), -ref[ct]);
        } else if (kMode == kCapped || a.softcap > 0.0f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fmaf(cap, tanh_of(y[j]), -ref[ct]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] -= ref[ct];
        }
      }
      if constexpr (kMode == kBiased) {
        const float at = (float)(pos[ct] - first);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = fmaf(-slope[ct], fabsf(at - (float)(16 * (j >> 2) + (j & 3))), y[j]);
      }
      if (masked) {
        const int end = min(limit[ct], key_end) - first;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 16 * (j >> 2) + (j & 3) < end ? y[j] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, y[j]);
      if (__ballot(top > most[ct])) {
        top = across_max(top);
        // a whole number, and none for columns whose own scores ask for none
        const bool moves = top > most[ct], first_one = most[ct] == -INFINITY;
        const float over = moves ? __builtin_ceilf(top) : 0.0f;
        ref[ct] += over;
        if (moves) most[ct] = kGrowth;
        // nothing has been summed where the first reference is taken
        const float f = first_one ? 1.0f : __builtin_amdgcn_exp2f(-over);
        l[ct] *= f;
        mean[ct] *= f;
        shrink(ct, first_one ? 0 : (int)fminf(over, 4096.0f));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] -= over;
      }
      // two loops, and not a branch in each turn of one
      if (!masked) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f32x4 vmul = step_of(nums, t, kg), vadd = mean_of(nums, t, kg);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float& z = y[4 * t + r];
            const float p = __builtin_amdgcn_exp2f(z);
            l[ct] += p;
            mean[ct] = fmaf(p, vadd[r], mean[ct]);
            z = p * vmul[r];
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const f32x4 vmul = step_of(nums, t, kg), vadd = mean_of(nums, t, kg);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float& z = y[4 * t + r];
            const float p = __builtin_amdgcn_exp2f(z);
            l[ct] += p;
            // what a column does not see may hold a NaN
            const bool seen = z != -INFINITY;
            mean[ct] = seen ? fmaf(p, vadd[r], mean[ct]) : mean[ct];
            z = seen ? p * vmul[r] : 0.0f;
          }
        }
      }
      float size = fabsf(y[0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) size = fmaxf(size, fabsf(y[j]));
      if (__ballot(size * per_unit[ct] > kMostWeight)) make_room(ct, size);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= per_unit[ct];
      w[ct] = __builtin_bit_cast(f16x8, u32x4{pack_f16(y[0], y[1]), pack_f16(y[2], y[3]),
                                              pack_f16(y[4], y[5]), pack_f16(y[6], y[7])});
    }
  }

  __device__ inline void add_values(int e, f16x8 x, const f16x8 (&w)[CT]) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
      o[ct][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w[ct], o[ct][e], 0, 0, 0);
  }
};

// N elements of column c from element `first` on: y with its sum and reference, as
// the result or as a piece's share.
template <typename T, int N>
__device__ inline void leave(const CachedArgs& a, const Work& w, int c, int first, float (&y)[N],
                             float sum, float top, bool number) {
  const int64_t token = w.d.qs + c / a.group;
  const int head = w.hk * a.group + c % a.group;
  if (a.whole) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] *= inv;
    store_elems((T*)(a.out + token * a.out_row + head * a.out_head + first), y);
    if (a.lse && number)
      a.lse[(int64_t)head * a.docs.rows_q + token] =
          sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  } else {
    const int64_t slot =
        ((int64_t)(a.first_piece + w.piece) * a.heads_q + head) * a.docs.rows_q + token;
    store_elems(a.part_o + slot * a.dim + first, y);
    if (number) {
      a.part_ml[2 * slot] = top;
      a.part_ml[2 * slot + 1] = sum;
    }
  }
}

// Few columns: 16 CT a workgroup, its wavefronts take the piece's keys in turn.
// With 16 it is the reading of the cache, with 32 its arithmetic weighs as much.  A
// tile is in flight in the registers that the one before has freed.
template <int DT>
struct FewMemory {
  f32x4 num[4][kNumbers / 4];
  float o[4][16][DT + 4], m[4][16], l[4][16], c[4][16];
};
template <typename T, int kBits, int DT, int CT, int kMode>
__device__ inline void few_columns(const CachedArgs& a, uint32_t block, FewMemory<DT>& mem) {
  typedef KeyCodes<T, kBits> K;
  typedef ValueCodes<kBits, DT> V;
  constexpr int kSteps = DT / 32, kElems = V::kElems;
  auto &s_o = mem.o;
  auto &s_m = mem.m, &s_l = mem.l, &s_c = mem.c;
  const int lane = threadIdx.x & 63, n = lane & 15, kg = lane >> 4;
  const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Work w;
  if (!find_work(a, block, 16 * CT, w)) return;
  float* const nums = (float*)mem.num[wave];
  const float to_log2 = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
  for (int col0 = w.first; col0 < w.end; col0 += 16 * CT) {
    const int last_col = min(col0 + 16 * CT, w.cols) - 1;
    const int all_see = key_limit(a, w.d, col0 / a.group);
    const int key_end = min((int)min((int64_t)w.d.kl, (int64_t)w.key0 + w.keys),
                            key_limit(a, w.d, last_col / a.group));
    int key = w.key0 + 32 * wave;
    // the first tile is on its way before the queries are looked at
    Tiles<T, kBits, DT> tile;
    tile.start(a, w, key, key_end);
    Columns<T, kBits, DT, CT, kMode> col;
    col.start(a, w, col0);
    for (; key < key_end; key += kStepKeys) {
      tile.leave_numbers(nums, to_log2);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      tile.load_numbers(key + kStepKeys);
      f32x4 s[2][CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) s[0][ct] = s[1][ct] = (f32x4)(0.0f);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const auto x = K::operand(tile.k.w[t] + i * kBits / 4);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) s[t][ct] = Mat16<T>::mul(x, col.q[ct][i], s[t][ct]);
        }
      tile.next_keys(key + kStepKeys);
      __builtin_amdgcn_sched_barrier(0);
      f16x8 p[CT];
      col.weigh(a, nums, s, key + 32 > all_see || key + 32 > key_end, key + 4 * kg,
                                key_end, p);
#pragma unroll
      for (int e = 0; e < kElems; ++e) col.add_values(e, V::operand(tile.v.w, e), p);
      tile.next_values(key + kStepKeys);
      __builtin_amdgcn_sched_barrier(0);
    }

    // The four wavefronts' sums, 16 columns at a time: 16 lanes a column.
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const float lsum = across_sum(col.l[ct]), msum = across_sum(col.mean[ct]);
      __syncthreads();
      if (kg == 0) {
        s_m[wave][n] = col.ref[ct];
        s_l[wave][n] = lsum;
        s_c[wave][n] = msum;
      }
#pragma unroll
      for (int e = 0; e < kElems; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          s_o[wave][n][V::element(4 * kg + r, e)] = col.o[ct][e][r] * 512.0f * col.unit(ct);
      __syncthreads();
      const int c16 = threadIdx.x >> 4, first = (threadIdx.x & 15) * kElems;
      const int c = col0 + 16 * ct + c16;
      if (c < w.cols && first < a.dim) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = s_l[i][c16] == 0.0f ? top : fmaxf(top, s_m[i][c16]);
        float sum = 0.0f, add = 0.0f, y[kElems];
#pragma unroll
        for (int e = 0; e < kElems; ++e) y[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (s_l[i][c16] == 0.0f) continue;
          const float f = __builtin_amdgcn_exp2f(s_m[i][c16] - top);
          sum = fmaf(f, s_l[i][c16], sum);
          add = fmaf(f, s_c[i][c16], add);
#pragma unroll
          for (int e = 0; e < kElems; ++e) y[e] = fmaf(f, s_o[i][c16][first + e], y[e]);
        }
#pragma unroll
        for (int e = 0; e < kElems; ++e) y[e] += add;
        leave<T>(a, w, c, first, y, sum, top, first == 0);
      }
    }
  }
}

// Many columns: 32 a wavefront, 128 a workgroup.  Each wavefront brings 32 of 128
// keys to operands, in LDS and in the order in which lanes read them, for all
// four: a quarter of the conversions that the few-column form would make.
constexpr int kManyCols = 128;
template <int DT>
struct ManyMemory {
  u32x4 k[4][DT / 16][64], v[4][DT / 16][64];
  f32x4 num[4][kNumbers / 4];
};
template <typename T, int kBits, int DT, int kMode>
__device__ inline void many_columns(const CachedArgs& a, uint32_t block, ManyMemory<DT>& mem) {
  typedef KeyCodes<T, kBits> K;
  typedef ValueCodes<kBits, DT> V;
  typedef typename Mat16<T>::V8 V8;
  constexpr int CT = 2, kSteps = DT / 32, kElems = V::kElems;
  auto &s_k = mem.k, &s_v = mem.v;
  const int lane = threadIdx.x & 63, n = lane & 15, kg = lane >> 4;
  const int wave = (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Work w;
  if (!find_work(a, block, kManyCols, w)) return;
  const float to_log2 = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
  for (int col0 = w.first; col0 < w.end; col0 += kManyCols) {
    const int last_col = min(col0 + kManyCols, w.cols) - 1;
    const int key_end = min((int)min((int64_t)w.d.kl, (int64_t)w.key0 + w.keys),
                            key_limit(a, w.d, last_col / a.group));
    // this wavefront's own columns, and the keys that all and any of them see
    const int mine = col0 + 16 * CT * wave, mine_last = min(mine + 16 * CT, w.cols) - 1;
    const bool idle = mine >= w.cols;
    const int all_see = idle ? 0 : key_limit(a, w.d, mine / a.group);
    const int any_sees = idle ? 0 : min(key_end, key_limit(a, w.d, mine_last / a.group));
    Tiles<T, kBits, DT> tile;
    tile.start(a, w, w.key0 + 32 * wave, key_end);
    Columns<T, kBits, DT, CT, kMode> col;
    col.start(a, w, mine);
    for (int base = w.key0; base < key_end; base += kStepKeys) {
      const int own = base + 32 * wave;
      // all have read the tiles before
      __syncthreads();
      tile.leave_numbers((float*)mem.num[wave], to_log2);
      tile.load_numbers(own + kStepKeys);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          s_k[wave][t * kSteps + i][lane] =
              __builtin_bit_cast(u32x4, K::operand(tile.k.w[t] + i * kBits / 4));
      tile.next_keys(own + kStepKeys);
#pragma unroll
      for (int e = 0; e < kElems; ++e)
        s_v[wave][e][lane] = __builtin_bit_cast(u32x4, V::operand(tile.v.w, e));
      tile.next_values(own + kStepKeys);
      __syncthreads();
#pragma unroll 1
      for (int sub = 0; sub < 4; ++sub) {
        const int key = base + 32 * sub;
        if (key >= any_sees) break;
        f32x4 s[2][CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) s[0][ct] = s[1][ct] = (f32x4)(0.0f);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const V8 x = __builtin_bit_cast(V8, s_k[sub][t * kSteps + i][lane]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) s[t][ct] = Mat16<T>::mul(x, col.q[ct][i], s[t][ct]);
          }
        f16x8 p[CT];
        col.weigh(a, (const float*)mem.num[sub], s, key + 32 > all_see || key + 32 > key_end,
                  key + 4 * kg, key_end, p);
#pragma unroll
        for (int e = 0; e < kElems; ++e)
          col.add_values(e, __builtin_bit_cast(f16x8, s_v[sub][e][lane]), p);
      }
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const float sum = across_sum(col.l[ct]), add = across_sum(col.mean[ct]);
      const int c = mine + 16 * ct + n;
      if (c >= w.cols || c >= w.end) continue;
      // a lane has a quarter of the column's elements, side by side
      float y[DT / 4];
#pragma unroll
      for (int e = 0; e < kElems; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          y[V::element(r, e)] = col.o[ct][e][r] * 512.0f * col.unit(ct) + add;
#pragma unroll
      for (int i = 0; i < DT / 4; i += 8) {
        const int first = kg * (DT / 4) + i;
        if (first >= a.dim) continue;
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = sum == 0.0f ? 0.0f : y[i + e];
        leave<T>(a, w, c, first, z, sum, sum == 0.0f ? -INFINITY : col.ref[ct], first == 0);
      }
    }
  }
}

template <typename T, int kBits, int DT, int CT, int kMode>
__global__ void __launch_bounds__(256, CT == 1 ? (DT == 64 ? 4 : 3) : 2)
    cached_few_kernel(CachedArgs a) {
  __shared__ FewMemory<DT> s_mem;
  few_columns<T, kBits, DT, CT, kMode>(a, a.block0 + blockIdx.x, s_mem);
}
template <typename T, int kBits, int DT, int kMode>
__global__ void __launch_bounds__(256, 2) cached_many_kernel(CachedArgs a) {
  __shared__ ManyMemory<DT> s_mem;
  many_columns<T, kBits, DT, kMode>(a, a.block0 + blockIdx.x, s_mem);
}

// Both passes in one launch, the shared keys' workgroups first: those of either hide
// what the other waits for (us with two launches : with one, caches from memory; 64
// requests behind 16,384 keys 54.5 : 48.0, 48 behind three prompts 31.0 : 22.6).
template <typename T, int kBits, int DT, int kMode>
__global__ void __launch_bounds__(256, 2) cached_both_kernel(CachedArgs own, CachedArgs shared) {
  __shared__ __align__(16) union {
    FewMemory<DT> few;
    ManyMemory<DT> many;
  } s_mem;
  static_assert(sizeof(CachedArgs) % alignof(CachedArgs) == 0 && alignof(CachedArgs) == 8,
                "one argument right after the other");
  const uint32_t block = own.block0 + blockIdx.x;
  const bool of_shared = block < shared.blocks;
  // Read where the launch has put them, one after the other: a choice between two
  // arguments would copy both into scratch memory (104 us for the first of these).  A
  // copy, since what is behind a pointer would be read again after each fence (91).
  typedef const __attribute__((address_space(4))) CachedArgs* Args;
  const CachedArgs a =
      *(const CachedArgs*)((Args)__builtin_amdgcn_kernarg_segment_ptr() + (of_shared ? 1 : 0));
  const uint32_t at = of_shared ? block : block - shared.blocks;
  if (a.width == 16) few_columns<T, kBits, DT, 1, kMode>(a, at, s_mem.few);
  else if (a.width == 32) few_columns<T, kBits, DT, 2, kMode>(a, at, s_mem.few);
  else many_columns<T, kBits, DT, kMode>(a, at, s_mem.many);
}

// A token's pieces of one head, and those of the keys it shares: kLanes lanes
// have the head's elements, four each, and the groups of so many lanes take
// pieces in turn; what they found meets in LDS.  A workgroup has one token, or all
// of a document of few.  kThreads is 64 where there are few pieces, else 256.  A
// launch and three dependent reads, 5 us; of large results the pieces' reading (4
// pieces of 1,024 tokens, 16 heads of 128: 34 MB in 12 us).
constexpr int kMostPieces = 256;  // of a pass
template <typename T, int kLanes, int kThreads>
__global__ void __launch_bounds__(kThreads) cached_join_kernel(CachedArgs a) {
  constexpr int kGroups = kThreads / kLanes, kWaves = kThreads / 64;
  __shared__ float s_f[2 * kMostPieces], s_top[kWaves], s_sum[kWaves];
  __shared__ __align__(16) f32x4 s_o[kGroups][kLanes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t block = a.block0 + blockIdx.x;
  const int head = (int)(block % (uint32_t)a.heads_q);
  uint32_t local = 0, units;
  Doc d;
  if (!a.looked_up) d = load_doc(a.docs, (int)(block / (uint32_t)a.heads_q));
  else if (find_document<false>(a.docs, 1, 1, block / (uint32_t)a.heads_q, &local, &units, &d) < 0)
    return;
  const int last = a.looked_up ? (int)local + 1 : d.ql;
  for (int t = (int)local; t < last; ++t) {
    const int64_t token = d.qs + t;
    const int size = piece_keys(d.kl, a.pieces, a.piece);
    const int own = max(1, (int)(((int64_t)d.kl + size - 1) / size));
    int more = 0;
    for (int base = 0; base < a.shared.count; base += 64) {
      Doc g = {0, 0, 0, 0, 0};
      if (base + lane < a.shared.count) g = load_doc(a.shared, base + lane);
      const uint64_t hit = __ballot(token >= g.qs && token < (int64_t)g.qs + g.ql);
      if (!hit) continue;
      const int kl = __builtin_amdgcn_readlane(g.kl, __ffsll((unsigned long long)hit) - 1);
      const int n = piece_keys(kl, a.pieces_shared, a.piece_shared);
      more = (int)(((int64_t)kl + n - 1) / n);
      break;
    }
    const int count = own + more;
    const auto slot = [&](int p) {
      const int at = p < own ? p : a.pieces + p - own;
      return ((int64_t)at * a.heads_q + head) * a.docs.rows_q + token;
    };
    // what each piece counts for: its sum times 2^(its reference - the largest)
    float top = -INFINITY;
    for (int p = threadIdx.x; p < count; p += kThreads) {
      const f32x2 ml = *(const f32x2*)(a.part_ml + 2 * slot(p));
      s_f[p] = ml.x;
      top = ml.y == 0.0f ? top : fmaxf(top, ml.x);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if (kWaves > 1) {
      if (lane == 0) s_top[wave] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) top = fmaxf(top, s_top[i]);
    }
    float sum = 0.0f;
    for (int p = threadIdx.x; p < count; p += kThreads) {
      const float l = a.part_ml[2 * slot(p) + 1];
      // a piece whose sum is zero holds zeros
      const float f = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(s_f[p] - top);
      s_f[p] = f;
      sum = fmaf(f, l, sum);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (kWaves > 1 && lane == 0) s_sum[wave] = sum;
    __syncthreads();
    if (kWaves > 1) {
      sum = s_sum[0];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) sum += s_sum[i];
    }
    const int group = threadIdx.x / kLanes, e = (threadIdx.x % kLanes) * 4;
    f32x4 x = (f32x4)(0.0f);
    if (e < a.dim) {
#pragma unroll 4
      for (int p = group; p < count; p += kGroups) {
        const f32x4 v = *(const f32x4*)(a.part_o + slot(p) * a.dim + e);
        const float f = s_f[p];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaf(f, v[i], x[i]);
      }
    }
    s_o[group][threadIdx.x % kLanes] = x;
    __syncthreads();
    if (group == 0 && e < a.dim) {
#pragma unroll
      for (int i = 1; i < kGroups; ++i) x += s_o[i][threadIdx.x];
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
      store_elems((T*)(a.out + token * a.out_row + head * a.out_head + e), y);
    }
    if (a.lse && threadIdx.x == 0)
      a.lse[(int64_t)head * a.docs.rows_q + token] =
          sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    __syncthreads();  // before LDS is the next token's
  }
}

namespace {

// How a pass is cut: columns of a workgroup, units, pieces of a document's keys.
struct Cut {
  int width;  // 16, 32 or kManyCols
  bool looked_up;
  int64_t units;
  int pieces, piece;
};
Cut cut_of(const gs_attention_config& cfg, const gs_documents& d, int64_t rows_q,
           int64_t rows_k) {
  Cut o = {};
  const int64_t group = cfg.heads_q / cfg.heads_k;
  const int64_t longest_q = d.max_q_len > 0 && d.max_q_len < rows_q ? d.max_q_len : rows_q;
  const int64_t longest_k = d.max_k_len > 0 && d.max_k_len < rows_k ? d.max_k_len : rows_k;
  // The form for many columns pays where documents have several times 128 (us, it : 32
  // columns; 1,024 tokens of one request, 16 heads of 128 over 4, 417 : 465), not up to
  // 128 (100 tokens of eight requests 91 : 31), and not yet just past that (500 of 16
  // requests, 8 heads of 64 over 4, 47 : 36).
  o.width = longest_q * group <= 16 ? 16 : longest_q * group <= 128 ? 32 : kManyCols;
  o.looked_up = longest_q * group > o.width;
  o.units = o.looked_up ? rows_q * group / o.width + d.count : d.count;
  // units that have work: documents end inside one, half way on average
  const int64_t busy = o.looked_up ? rows_q * group / o.width + (d.count + 1) / 2 : d.count;
  const int64_t base = (busy > 0 ? busy : 1) * cfg.heads_k;
  // Workgroups wanted (all figures with caches from memory).  16 columns: two a compute
  // unit where there are few documents (four caches of 120,001 keys in all: 43, 46, 48,
  // 49 us with 512, 768, 1,024, 1,536), more where many of uneven length hide each
  // other's ends (64 caches of 100,003 keys, 8 heads of 64 in 4 bits: 40, 40, 40, 37, and
  // 35 with 2,048).  32 columns: in between (24 requests of a few tokens, 30,011 keys:
  // 26, 24, 23, 27 with 256, 512, 704, 1,024).  Many: what the chip holds at a time (the
  // 1,024 tokens: 788, 417, 497, 429 with 256, 512, 768, 1,024).
  const int64_t target = o.width == 16 ? (base >= 256 ? 1536 : 512) : o.width == 32 ? 704 : 512;
  int64_t pieces = (target + base - 1) / base;
  if (pieces > kMostPieces) pieces = kMostPieces;
  // Where the caller says how long documents are, all pieces have that share of the
  // longest.  Up to 2,048 keys, since documents of uneven length need pieces that
  // end together (64 caches of 524,288 keys in all: 137 us without that limit, 123,
  // 114, 114, 123 with 4,096, 2,048, 1,024, 512).
  int64_t piece = 2 * kStepKeys;
  if (d.max_k_len > 0) {
    piece = (longest_k + pieces - 1) / pieces;
    if (o.width == 16 && piece > 2048) piece = 2048;
    piece = (piece + kStepKeys - 1) / kStepKeys * kStepKeys;
    if (piece < 2 * kStepKeys) piece = 2 * kStepKeys;
    // workgroups without work cost little, but not nothing: 2^15 at most, where the
    // target asks for no more
    const int64_t room = (1 << 15) / base;
    pieces = pieces > room ? pieces : room < kMostPieces ? room : kMostPieces;
  }
  const int64_t most = (longest_k + piece - 1) / piece;
  if (pieces > most) pieces = most;
  o.pieces = (int)(pieces < 1 ? 1 : pieces);
  o.piece = (int)piece;
  return o;
}

struct Plan {
  Cut own, shared;
  bool whole;
  int64_t slots;
};
Plan plan_of(const gs_attention_config& cfg, const gs_documents& d, const gs_documents* shared,
             int64_t rows_q, int64_t rows_k) {
  Plan p = {};
  p.own = cut_of(cfg, d, rows_q, rows_k);
  if (shared && shared->count > 0) p.shared = cut_of(cfg, *shared, rows_q, rows_k);
  p.whole = p.own.pieces == 1 && p.shared.pieces == 0;
  p.slots = p.whole ? 0 : (int64_t)(p.own.pieces + p.shared.pieces) * cfg.heads_q * rows_q;
  return p;
}

size_t ml_bytes(const Plan& p) { return ((size_t)p.slots * 8 + 255) / 256 * 256; }

// Arguments of a pass; its workgroups.
int64_t set_pass(CachedArgs& a, const Cut& c) {
  a.pieces = c.pieces;
  a.piece = c.piece;
  a.looked_up = c.looked_up;
  a.width = c.width;
  a.units = (uint32_t)c.units;
  return (c.units * c.pieces + 7) / 8 * 8 * a.heads_k;
}

template <typename T, int kBits, int DT, int kMode>
hipError_t pass(CachedArgs a, const Cut& c, hipStream_t s) {
  return launch_all(set_pass(a, c), 256, [&](uint32_t first, dim3 n) {
    a.block0 = first;
    if (c.width == 16) cached_few_kernel<T, kBits, DT, 1, kMode><<<n, 256, 0, s>>>(a);
    else if (c.width == 32) cached_few_kernel<T, kBits, DT, 2, kMode><<<n, 256, 0, s>>>(a);
    else cached_many_kernel<T, kBits, DT, kMode><<<n, 256, 0, s>>>(a);
  });
}

template <typename T, int kBits, int DT, int kMode>
hipError_t run(const CachedArgs& a, const Plan& p, const Docs& shared, hipStream_t s) {
  hipError_t e;
  if (kMode != kBiased && p.shared.pieces > 0) {
    CachedArgs own = a, b = a;
    b.docs = shared;
    b.causal = 0;
    b.first_piece = p.own.pieces;
    const int64_t blocks = set_pass(b, p.shared);
    b.blocks = (uint32_t)blocks;
    e = launch_all(blocks + set_pass(own, p.own), 256, [&](uint32_t first, dim3 n) {
      own.block0 = first;
      cached_both_kernel<T, kBits, DT, kMode == kBiased ? kPlain : kMode><<<n, 256, 0, s>>>(own, b);
    });
  } else {
    e = pass<T, kBits, DT, kMode>(a, p.own, s);
  }
  if (e != hipSuccess || p.whole) return e;
  CachedArgs j = a;
  j.shared = shared;
  j.looked_up = p.own.looked_up;
  j.pieces = p.own.pieces;
  j.piece = p.own.piece;
  j.piece_shared = p.shared.piece;
  j.pieces_shared = p.shared.pieces;
  // with up to 16 pieces a wavefront has them in a few loads
  const int threads = p.own.pieces + p.shared.pieces <= 16 ? 64 : 256;
  const int64_t units = j.looked_up ? a.docs.rows_q : a.docs.count;
  return launch_all(units * a.heads_q, threads, [&](uint32_t first, dim3 n) {
    j.block0 = first;
    constexpr int kLanes = DT / 4;
    if (threads == 64) cached_join_kernel<T, kLanes, 64><<<n, 64, 0, s>>>(j);
    else cached_join_kernel<T, kLanes, 256><<<n, 256, 0, s>>>(j);
  });
}

template <typename T, int kBits, int DT>
hipError_t run(const CachedArgs& a, const Plan& p, const Docs& shared, hipStream_t s) {
  if (a.slopes) return run<T, kBits, DT, kBiased>(a, p, shared, s);
  if (a.softcap > 0.0f) return run<T, kBits, DT, kCapped>(a, p, shared, s);
  return run<T, kBits, DT, kPlain>(a, p, shared, s);
}

template <typename T>
hipError_t run(const CachedArgs& a, const Plan& p, const Docs& shared, int bits, hipStream_t s) {
  if (bits == 8)
    return a.dim <= 64 ? run<T, 8, 64>(a, p, shared, s) : run<T, 8, 128>(a, p, shared, s);
  return a.dim <= 64 ? run<T, 4, 64>(a, p, shared, s) : run<T, 4, 128>(a, p, shared, s);
}

}  // namespace
}  // namespace gs

extern "C" {

size_t gs_cached_attention_bytes(const gs_attention_config& cfg, const gs_documents& d,
                                 const gs_documents* shared, int64_t rows_q, int64_t rows_k) {
  const gs::Plan p = gs::plan_of(cfg, d, shared, rows_q, rows_k);
  return p.whole ? 0 : gs::ml_bytes(p) + (size_t)p.slots * cfg.head_dim * 4;
}

hipError_t gs_launch_cached_attention(const gs_attention_config& cfg, const gs_documents& d,
                                      const gs_documents* shared, int64_t rows_q, int64_t rows_k,
                                      const gs_heads& q, const gs_codes& k, const gs_codes& v,
                                      const gs_heads& out, float* lse, void* workspace,
                                      hipStream_t s) {
  const gs::Plan p = gs::plan_of(cfg, d, shared, rows_q, rows_k);
  gs::CachedArgs a = {};
  a.docs = gs::make_docs(d, rows_q, rows_k);
  gs::Docs more = {};
  if (shared) more = gs::make_docs(*shared, rows_q, rows_k);
  more.prefix = nullptr;  // all tokens see all shared keys
  a.heads_q = cfg.heads_q;
  a.heads_k = cfg.heads_k;
  a.group = cfg.heads_q / cfg.heads_k;
  a.dim = cfg.head_dim;
  a.causal = cfg.causal;
  a.scale = cfg.scale;
  a.softcap = cfg.softcap;
  a.slopes = cfg.slopes;
  a.q = (const uint16_t*)q.data; a.q_row = q.row; a.q_head = q.head;
  a.kc = (const uint8_t*)k.codes; a.kc_row = k.row; a.kc_head = k.head;
  a.vc = (const uint8_t*)v.codes; a.vc_row = v.row; a.vc_head = v.head;
  a.klow = k.low; a.kstep = k.step; a.k_ld = k.ld;
  a.vlow = v.low; a.vstep = v.step; a.v_ld = v.ld;
  a.out = (uint16_t*)out.data; a.out_row = out.row; a.out_head = out.head;
  a.lse = lse;
  a.whole = p.whole;
  a.part_ml = (float*)workspace;
  a.part_o = (float*)((char*)workspace + gs::ml_bytes(p));
  if (cfg.dtype == GS_BF16) return gs::run<gs::Bf16>(a, p, more, k.bits, s);
  return gs::run<gs::F16>(a, p, more, k.bits, s);
}

}  // extern "C"
