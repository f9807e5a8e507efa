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
  int parts;          // dk, dv: sums per query head
  int pieces, piece;  // few-column form: pieces of a document's keys, keys of one
  int tiles;          // few-column form: column tiles of a key head in the grid
  int pieces_last;    // few-column form: the order of the grid
  int col_units;      // few-column form: column tiles are units of the grid
  float* part_ml;     // [pieces][heads_q][rows_q][2]
  float* part_o;      // [pieces][heads_q][rows_q][dim]
  uint32_t block0;    // first workgroup of the launch
};

__device__ inline uint32_t block_of(const AttnArgs& a) { return a.block0 + blockIdx.x; }

constexpr int kKeys = 64;  // keys of a staged tile
constexpr int kCols = 128; // columns of a workgroup: four wavefronts of 32
constexpr int kRows = 32;  // query rows of a staged tile of the dk, dv kernel
constexpr int kPieceKeys = 128;  // one-token form: keys the four wavefronts take at a time

// How scores are made: kMode bits.
constexpr int kCap = 1;      // capped by tanh
constexpr int kGeneral = 2;  // distance bias, or a scale that is not positive
constexpr int kWide = 4;     // a cap far above most scores (with the other two)

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

// Byte offsets of this lane's operand reads in a staged tile.  Within a row the
// place of a chunk is its number XOR a few bits of the row, so every other
// read of a tile is these offsets XOR a constant (contraction step, column
// tile) plus a constant (row tile): few registers hold addresses.
template <int DT>
struct Lane {
  int rows;         // row lane % 32, chunk half
  int cols0, cols8; // transposing read: rows 4 half + (lane % 16) / 4 and 8 on
  __device__ inline Lane() {
    const int lane = threadIdx.x & 63;
    rows = 2 * place<DT>(lane & 31, lane >> 5);
    const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int d = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    cols0 = 2 * (place<DT>(r, d >> 3) + (d & 7));
    cols8 = 2 * (place<DT>(r + 8, d >> 3) + (d & 7));
  }
};

// Left or right operand: rows lane % 32 of the 32-row tile at byte `base` plus
// the lane's offset, contraction 16 ks + 8 half ...
template <typename T, int DT>
__device__ inline typename Mat<T>::V8 read_rows(const char* mem, int at, int r0, int ks) {
  const u32x4 w = *(const u32x4*)(mem + (at ^ (32 * ks)) + 2 * r0 * DT);
  return __builtin_bit_cast(typename Mat<T>::V8, w);
}

// Left operand of the transposed tile: rows are elements 32 dt + lane % 32,
// contraction slots the tile's rows r0 + 8 (j / 4) + 4 half + j % 4.
template <typename T, int DT>
__device__ inline typename Mat<T>::V8 read_cols(const char* mem, int at0, int at8, int r0, int dt) {
  typedef __attribute__((address_space(3))) s16x4 L;
  const s16x4 a =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(mem + (at0 ^ (64 * dt)) + 2 * r0 * DT));
  const s16x4 b =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(mem + (at8 ^ (64 * dt)) + 2 * r0 * DT));
  const s16x8 w = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(typename Mat<T>::V8, w);
}

// Eight results of a 32-row tile (registers 8 ks ...) as the right operand's
// 16 contraction slots.  Here softmax weights and score gradients are rounded
// to the type, since the matrix instruction takes no wider operand: the sums
// over them stay fp32, and what it adds is of the size of the inputs' and the
// outputs' own roundings (against 64 bits, outputs and gradients are off by 1.15
// to 1.45 times what a form in 32 bits, rounded at the end, is).  A second
// product for what the rounding leaves out would make the forward's matrix work
// half as much again.
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

// A tile of ROWS rows, copied from memory into LDS by all 256 lanes without
// passing through registers (buffer loads with an LDS destination: lane l of a
// wavefront fills the 16 bytes l of its kilobyte, so it is the source address
// that follows the tile's chunk order).  The buffer descriptor ends with the
// document's last row: rows past `valid` (and elements past dim, whose offset
// is past every end) arrive as zeros, without a branch; rows of a tile are
// within 2^31 bytes of each other (row strides are below 2^23 elements).
// The copies are counted by vmcnt but unknown to the compiler, whose own waits
// can only be longer for it: arrived() must come before the barrier after
// which the tile is read.
template <int DT, int ROWS>
__device__ inline void copy_tile(const char* mem, int tile, const uint16_t* base,
                                 int64_t row_stride, int valid, int dim) {
  constexpr int kChunks = DT / 8, kStep = 256 / kChunks;  // rows a pass
  static_assert(ROWS % kStep == 0 && kStep % 16 == 0, "a pass keeps the chunk order");
  const int stride = (int)row_stride * 2;
  const int64_t bytes = valid > 0 ? (int64_t)(valid - 1) * stride + dim * 2 : 0;
  const uint64_t address = (uint64_t)base;
  const i32x4 rsrc = {(int)address, (int)((address >> 32) & 0xffff),
                      (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00027000};
  const int r = threadIdx.x / kChunks;
  // place() moves chunk c of row r by an exclusive or, its own inverse
  const int c = (place<DT>(r, threadIdx.x % kChunks) - r * DT) / 8;
  uint32_t at = c * 8 < dim ? (uint32_t)(r * stride + c * 16) : 0x80000000u;
  const uint32_t lds =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(
                                         __attribute__((address_space(3))) const char*)mem +
                                     tile + (threadIdx.x >> 6) * 1024);
#pragma unroll
  for (int i = 0; i < ROWS / kStep; ++i) {
    asm volatile(
        "s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(at),
        "s"(rsrc), "s"(lds + i * 4096)
        : "memory", "m0");
    at = c * 8 < dim ? at + (uint32_t)(kStep * stride) : at;
  }
}
__device__ inline void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Thirty-two rows as operand fragments straight from memory (row lane % 32,
// elements 16 ks + 8 half ...), zeros past `valid` rows and dim elements; and
// their place in a staged tile.
template <typename T, int DT>
struct Fragments {
  typename Mat<T>::V8 f[DT / 16];
  __device__ inline void load(const uint16_t* base, int64_t row_stride, int valid, int dim) {
    const int stride = (int)row_stride * 2;
    const int64_t bytes = valid > 0 ? (int64_t)(valid - 1) * stride + dim * 2 : 0;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(base), 0, (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff),
        0x00027000);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int at = (lane & 31) * stride + half * 16;
#pragma unroll
    for (int ks = 0; ks < DT / 16; ++ks) {
      const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(
          rsrc, 16 * ks + 8 * half < dim ? at + 32 * ks : (int)0x80000000, 0, 0);
      f[ks] = __builtin_bit_cast(typename Mat<T>::V8, w);
    }
  }
  __device__ inline void store(char* mem, int tile, const Lane<DT>& at) const {
#pragma unroll
    for (int ks = 0; ks < DT / 16; ++ks)
      *(u32x4*)(mem + ((at.rows + tile) ^ (32 * ks))) = __builtin_bit_cast(u32x4, f[ks]);
  }
  __device__ inline f32x16 times(const typename Mat<T>::V8 (&b)[DT / 16]) const {
    f32x16 s = (f32x16)(0.0f);
#pragma unroll
    for (int ks = 0; ks < DT / 16; ++ks) s = Mat<T>::mul(f[ks], b[ks], s);
    return s;
  }
};

// What a wavefront wrote to its own LDS is there for its next reads.
__device__ inline void own_lds_written() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Dot product of two fragment columns, both halves together.
template <typename T, int N>
__device__ inline float dot_cols(const typename Mat<T>::V8 (&x)[N],
                                 const typename Mat<T>::V8 (&y)[N]) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf((float)x[i][j], (float)y[i][j], sum);
  return both_sum(sum);
}

// Four wavefronts' accumulators of 32 columns into LDS, for their sum.
template <int DT>
__device__ inline void leave_cols(float* s_raw, const f32x16 (&o)[DT / 32]) {
  constexpr int kStride = DT + 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 x = {o[dt][4 * i], o[dt][4 * i + 1], o[dt][4 * i + 2], o[dt][4 * i + 3]};
      *(f32x4*)(s_raw + (wave * 32 + (lane & 31)) * kStride + dt * 32 + 8 * i + 4 * (lane >> 5)) =
          x;
    }
  }
}

// N steps of a product whose operand `read(n)` comes from LDS: each read is
// issued A steps before its use (an LDS read takes about as long as four of the
// instructions it feeds), and the barriers keep the compiler from moving every
// read to the front, which costs more registers than there are.  prime() may
// stand well before run(), to have the first reads under way.
template <typename V, int N, int A>
struct Pipeline {
  V x[A + 1];
  template <typename Read>
  __device__ inline void prime(Read read) {
#pragma unroll
    for (int n = 0; n < A && n < N; ++n) x[n] = read(n);
  }
  template <typename Read, typename Use>
  __device__ inline void run(Read read, Use use) {
    // while the matrix unit is fed, this wavefront goes before others that are
    // at their scores
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (n + A < N) x[(n + A) % (A + 1)] = read(n + A);
      use(n, x[n % (A + 1)]);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  }
};

// s0 = tile at byte t0 times f0, s1 = tile at byte t1 times f1 (32 rows each,
// taken in turn so that no instruction waits for the one before it).
template <typename T, int DT, int A = 3>
__device__ inline void two_products(const char* mem, int t0, int t1, const Lane<DT>& at,
                                    const typename Mat<T>::V8 (&f0)[DT / 16],
                                    const typename Mat<T>::V8 (&f1)[DT / 16], f32x16& s0,
                                    f32x16& s1) {
  typedef typename Mat<T>::V8 V8;
  const int a0 = at.rows + t0, a1 = at.rows + t1;
  Pipeline<V8, DT / 8, A> p;
  auto read = [&](int n) { return read_rows<T, DT>(mem, n & 1 ? a1 : a0, 0, n >> 1); };
  s0 = s1 = (f32x16)(0.0f);
  p.prime(read);
  p.run(read, [&](int n, const V8& x) {
    if (n & 1) s1 = Mat<T>::mul(x, f1[n >> 1], s1);
    else s0 = Mat<T>::mul(x, f0[n >> 1], s0);
  });
}

// The same with the second product's right operand in LDS too (byte right).
template <typename T, int DT, int A>
__device__ inline void two_products_staged(const char* mem, int t0, int t1, int right,
                                           const Lane<DT>& at,
                                           const typename Mat<T>::V8 (&f0)[DT / 16], f32x16& s0,
                                           f32x16& s1) {
  typedef typename Mat<T>::V8 V8;
  struct Pair {
    V8 x, y;
  };
  const int a0 = at.rows + t0, a1 = at.rows + t1, r = at.rows + right;
  Pipeline<Pair, DT / 8, A> p;
  auto read = [&](int n) {
    Pair o;
    o.x = read_rows<T, DT>(mem, n & 1 ? a1 : a0, 0, n >> 1);
    if (n & 1) o.y = read_rows<T, DT>(mem, r, 0, n >> 1);
    return o;
  };
  s0 = s1 = (f32x16)(0.0f);
  p.prime(read);
  p.run(read, [&](int n, const Pair& v) {
    if (n & 1) s1 = Mat<T>::mul(v.x, v.y, s1);
    else s0 = Mat<T>::mul(v.x, f0[n >> 1], s0);
  });
}

// o += (32 R rows from byte `tile`, transposed) times the R tiles of p.
template <typename T, int DT, int R, int A = 3>
struct AddCols {
  typedef typename Mat<T>::V8 V8;
  static constexpr int M = DT / 32;
  Pipeline<V8, 2 * M * R, A> p;
  const char* mem;
  int a, b;
  __device__ inline V8 read(int n) const {
    return read_cols<T, DT>(mem, a, b, n / M * 16, n % M);
  }
  __device__ inline AddCols(const char* mem, int tile, const Lane<DT>& at)
      : mem(mem), a(at.cols0 + tile), b(at.cols8 + tile) {
    p.prime([&](int n) { return read(n); });
  }
  __device__ inline void run(const f32x16 (&s)[R], f32x16 (&o)[DT / 32]) {
    V8 w[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) w[i] = pack_cols<T>(s[i / 2], i % 2);
    run(w, o);
  }
  __device__ inline void run(const V8 (&w)[2 * R], f32x16 (&o)[DT / 32]) {
    p.run([&](int n) { return read(n); },
          [&](int n, const V8& x) { o[n % M] = Mat<T>::mul(x, w[n / M], o[n % M]); });
  }
  // two sums at once
  __device__ inline void run(const f32x16& s0, f32x16 (&o0)[DT / 32], const f32x16& s1,
                             f32x16 (&o1)[DT / 32]) {
    static_assert(R == 1, "one tile of rows");
    const V8 w0[2] = {pack_cols<T>(s0, 0), pack_cols<T>(s0, 1)};
    const V8 w1[2] = {pack_cols<T>(s1, 0), pack_cols<T>(s1, 1)};
    p.run([&](int n) { return read(n); }, [&](int n, const V8& x) {
      o0[n % M] = Mat<T>::mul(x, w0[n / M], o0[n % M]);
      o1[n % M] = Mat<T>::mul(x, w1[n / M], o1[n % M]);
    });
  }
};

// Constants of the scores, in units of log2.
struct Scale {
  float mul, cap_in, cap_out;
};
template <int kMode>
__device__ inline Scale scale_of(const AttnArgs& a) {
  Scale c;
  c.mul = a.scale * kLog2e;
  c.cap_in = kMode & kCap ? a.scale / a.softcap : 0.0f;
  c.cap_out = a.softcap * kLog2e;
  return c;
}

// A raw product as a score, less `away` = slope |i' - j|; f receives
// 1 - tanh^2.  Plain scores stay raw (their factor mul is applied with the
// subtraction that follows).
template <int kMode, typename Away>
__device__ inline float score(float s, const Scale& c, Away away, float& f) {
  f = 1.0f;
  if constexpr (kMode == 0) return s;
  float x;
  if constexpr (kMode & kCap) {
    const float th = kMode & kWide ? tanh_wide(s * c.cap_in) : tanh_of(s * c.cap_in);
    f = fmaf(-th, th, 1.0f);
    x = th * c.cap_out;
  } else {
    x = s * c.mul;
  }
  if constexpr (kMode & kGeneral) x -= away();
  return x;
}

// Four results of 16 as they are stored: rows 8 i + 4 half + j of the
// transposed output, i.e. four consecutive elements of the lane's column.
template <typename T, int DT, typename F>
__device__ inline void store_col(uint16_t* p, int dim, F value) {
  const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = dt * 32 + 8 * i + 4 * half;
      if (e < dim) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = value(dt, 4 * i + j);
        store_elems((T*)(p + e), x);
      }
    }
  }
}

// A query column of this lane.
struct Col {
  int token, head, pos, lim;
  bool ok;
};
__device__ inline Col column(const AttnArgs& a, const Doc& d, int hk, uint32_t c, uint32_t cols) {
  Col o;
  o.ok = c < cols;
  o.token = (int)(c / a.group);
  o.head = hk * a.group + (int)(c % a.group);
  o.pos = o.token + d.kl - d.ql;
  o.lim = key_limit(a, d, o.token);
  return o;
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// The same value, unknown to the compiler.  Taken inside a uniform branch it
// keeps what depends on it there: masks are needed in few tiles, and the
// compiler would rather select in all of them (104 of the forward's 233 vector
// instructions a tile).
__device__ inline int only_here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The running softmax of a column over N 32-key tiles of scores.
template <int N>
__device__ inline void mask_scores(f32x16 (&s)[N], int room) {
  const int here = only_here(room);
#pragma unroll
  for (int rt = 0; rt < N; ++rt)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[rt][i] = rt * 32 + result_row(i) < here ? s[rt][i] : -INFINITY;
}
template <int N>
__device__ inline float highest(const f32x16 (&s)[N]) {
  float top = -INFINITY;
#pragma unroll
  for (int rt = 0; rt < N; ++rt)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[rt][i]);
  return both_max(top);
}
// Moves the reference m where a score passes it by more than 8: weights then
// stay below 2^8, far inside every type, and the accumulators are rarely
// rescaled.
template <int DT, int N>
__device__ inline void move_reference(float top, float& m, float& l, f32x16 (&o)[DT / 32]) {
  if (__any(top > m + 8.0f)) {
    const float now = fmaxf(m, top);
    const float alpha = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - now);
    l *= alpha;
#pragma unroll
    for (int i = 0; i < DT / 32; ++i) o[i] *= alpha;
    m = now;
  }
}
__device__ inline void weights_of(f32x16& s, float mul, float ref, float& l) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], mul, -ref));
    l += s[i];
  }
}
template <int DT, int N>
__device__ inline void softmax_step(f32x16 (&s)[N], float mul, bool masked, int k0, int lim,
                                    float& m, float& l, f32x16 (&o)[DT / 32]) {
  if (masked) mask_scores(s, lim - k0);
  move_reference<DT, N>(highest(s) * mul, m, l, o);
  const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int rt = 0; rt < N; ++rt) weights_of(s[rt], mul, ref, l);
}

// Scores of one 32-key tile in place.
template <int kMode>
__device__ inline void make_scores(f32x16& s, const Scale& c, float slope, int off) {
  if constexpr (kMode != 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float f;
      s[i] = score<kMode>(s[i], c,
                          [&] { return slope * fabsf((float)(off - result_row(i))); }, f);
    }
  }
}

// A workgroup takes 128 columns, a wavefront 32; key and value tiles of 64
// pass through LDS, copied there one tile ahead of their use.  Two workgroups
// share a compute unit, one's matrix instructions beside the other's
// exponentials.  (The next tile's products and this one's exponentials
// interleaved in one instruction stream were no faster with 128-element heads
// and a sixth slower with 64; nor were workgroups of eight wavefronts, which
// copy each tile half as often.)
// Bound by issue: the matrix unit is busy 47% of the time and the vector ALU
// 46%, with the two workgroups' phases seldom apart.  One causal document of
// 16,384 tokens, 16 bf16 heads of 128 over 4: 1.06 ms, 1.03 PFLOP/s of the pairs
// that are seen, where a large matrix product reaches 1.6.
template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, 2) void attention_fwd_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  // two buffers of a key and a value tile each
  constexpr int kTile = kKeys * DT * 2;
  __shared__ __align__(256) char mem[4 * kTile];
  const Lane<DT> at;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hk = block_of(a) % a.heads_k;
  uint32_t local, units;
  Doc d;
  if (find_document<false>(a.docs, a.group, kCols, block_of(a) / a.heads_k, &local, &units, &d) < 0)
    return;
  // long causal rows first
  const uint32_t col0 = (units - 1 - local) * kCols;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const int last_token = (int)((min(col0 + kCols, cols) - 1) / a.group);
  const int end = key_limit(a, d, last_token);
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  auto copy = [&](int k0, int to) {
    copy_tile<DT, kKeys>(mem, to, kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
    copy_tile<DT, kKeys>(mem, to + kTile, vb + (int64_t)k0 * a.v_row, a.v_row, d.kl - k0, a.dim);
  };
  if (end > 0) copy(0, 0);
  const Col col = column(a, d, hk, col0 + wave * 32 + (lane & 31), cols);
  const int64_t row = d.qs + col.token;
  V8 qf[DT / 16];
  load_cols<T, DT>(a.q + row * a.q_row + (int64_t)col.head * a.q_head, col.ok, a.dim, qf);
  const Scale sc = scale_of<kMode>(a);
  const float mul = kMode == 0 ? sc.mul : 1.0f;
  const float slope = (kMode & kGeneral) && a.slopes && col.ok ? a.slopes[col.head] * kLog2e
                                                               : 0.0f;
  f32x16 o[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) o[i] = (f32x16)(0.0f);
  float m = -INFINITY, l = 0.0f;
  const int wave_lo = __builtin_amdgcn_readlane(col.lim, 0);
  const int wave_hi = min(__builtin_amdgcn_readlane(col.lim, 31), end);
  int buf = 0;
  for (int k0 = 0; k0 < end; k0 += kKeys, buf ^= 2 * kTile) {
    arrived();
    __syncthreads();
    if (k0 + kKeys < end) copy(k0 + kKeys, buf ^ (2 * kTile));
    if (k0 >= wave_hi) continue;
    f32x16 s[2];
    two_products<T, DT>(mem, buf, buf + kTile / 2, at, qf, qf, s[0], s[1]);
    AddCols<T, DT, 2> add(mem, buf + kTile, at);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
      make_scores<kMode>(s[rt], sc, slope, col.pos - k0 - rt * 32);
    softmax_step<DT, 2>(s, mul, k0 + kKeys > wave_lo, k0, col.lim, m, l, o);
    add.run(s, o);
  }
  const float sum = both_sum(l);
  if (!col.ok) return;
  const bool none = col.lim <= 0;
  const float inv = none || sum == 0.0f ? 0.0f : 1.0f / sum;
  store_col<T, DT>(a.out0 + row * a.out0_row + (int64_t)col.head * a.out0_head, a.dim,
                   [&](int dt, int i) { return none ? 0.0f : o[dt][i] * inv; });
  if (a.lse && lane < 32)
    a.lse[(int64_t)col.head * a.docs.rows_q + row] =
        none ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Few columns in all: the keys are what there is to split.  A workgroup takes
// 32 columns of a key head and one piece of their document's keys, its four
// wavefronts 32 keys each in turn.  Keys come straight from memory as the left
// operand, values pass through the wavefront's own LDS for the transposing
// read, and both are on their way for the next tile while this one is
// computed.  The wavefronts' results are joined in LDS; where a document has
// several pieces, attention_join_kernel joins those.  One-token requests (all
// of a key head's query heads are columns) have one column tile a document;
// otherwise (col_units) the document of a column tile is looked up.  One-token
// calls are bound by reading the caches: 246 MB of four documents 45 us and 6 to
// join with the caches held on the chip, 63 in all from memory (3.9 TB/s, what a
// sum of a large tensor reaches).
struct StepItem {
  int hk, piece;
  uint32_t col0;
  bool none;
  Doc d;
};
__device__ inline StepItem step_item(const AttnArgs& a, int u) {
  StepItem o;
  o.hk = u % a.heads_k;
  u /= a.heads_k;
  // With many documents, all first pieces before all second ones: documents
  // have different numbers of them, and workgroups are dealt to the compute
  // units in turn, so that with four pieces a document every fourth unit would
  // get all the fourth ones.  With few, a document's pieces in a row.
  if (a.pieces_last) {
    o.piece = u / a.tiles;
    u %= a.tiles;
  } else {
    o.piece = u % a.pieces;
    u /= a.pieces;
  }
  o.col0 = 0;
  o.none = false;
  if (a.col_units) {
    uint32_t local = 0, units = 1;
    o.none = find_document<false>(a.docs, a.group, 32, u, &local, &units, &o.d) < 0;
    o.col0 = (units - 1 - local) * 32;  // long causal rows first
  } else {
    o.d = load_doc(a.docs, u);
  }
  return o;
}
__device__ inline int pieces_of(const AttnArgs& a, const Doc& d) {
  return max(1, min(a.pieces, (int)(((uint32_t)d.kl + a.piece - 1) / (uint32_t)a.piece)));
}

template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, DT == 128 ? 2 : 3) void attention_step_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  constexpr int kChunks = DT / 8;
  constexpr int kPer = 32 * kChunks / 64;
  constexpr int kStride = DT + 4;
  // the values' tiles, and after the loop the wavefronts' results
  __shared__ __align__(256) float s_raw[4 * 32 * kStride];
  __shared__ float s_m[4][32], s_l[4][32];
  char* const mem = (char*)s_raw;
  const int tile = (threadIdx.x >> 6) * 32 * DT * 2;
  const Lane<DT> at_lane;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const StepItem it = step_item(a, block_of(a));
  if (it.none) return;
  const Doc& d = it.d;
  const int hk = it.hk, piece = it.piece, pieces = pieces_of(a, d);
  if (piece >= pieces) return;
  const int key_lo = piece * a.piece;
  const int key_hi = piece == pieces - 1 ? d.kl : key_lo + a.piece;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  const Scale sc = scale_of<kMode>(a);
  const float mul = kMode == 0 ? sc.mul : 1.0f;
  for (uint32_t col0 = it.col0; col0 < cols; col0 += 32) {
    const Col col = column(a, d, hk, col0 + (lane & 31), cols);
    V8 qf[DT / 16];
    load_cols<T, DT>(a.q + (int64_t)(d.qs + col.token) * a.q_row + (int64_t)col.head * a.q_head,
                     col.ok, a.dim, qf);
    const float slope = (kMode & kGeneral) && a.slopes && col.ok ? a.slopes[col.head] * kLog2e
                                                                 : 0.0f;
    const int last_token = (int)((min(col0 + 32, cols) - 1) / a.group);
    const int end = min(key_hi, key_limit(a, d, last_token));
    const int wave_lo = __builtin_amdgcn_readlane(col.lim, 0);
    f32x16 o[DT / 32];
#pragma unroll
    for (int i = 0; i < DT / 32; ++i) o[i] = (f32x16)(0.0f);
    float m = -INFINITY, l = 0.0f;
    Fragments<T, DT> kf;
    u32x4 vw[kPer];
    auto fetch = [&](int k0) {
      kf.load(kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
      const int stride = (int)a.v_row * 2;
      const int64_t bytes = (int64_t)(d.kl - k0 - 1) * stride + a.dim * 2;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(vb + (int64_t)k0 * a.v_row), 0,
          (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff), 0x00027000);
      const int r = lane / kChunks, c = lane % kChunks;
      uint32_t at = c * 8 < a.dim ? (uint32_t)(r * stride + c * 16) : 0x80000000u;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        vw[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)at, 0, 0);
        at = c * 8 < a.dim ? at + (uint32_t)(64 / kChunks * stride) : at;
      }
    };
    int k0 = key_lo + wave * 32;
    if (k0 < end) fetch(k0);
    for (; k0 < end; k0 += kPieceKeys) {
      f32x16 s[1] = {kf.times(qf)};
      // the wavefront's own tile: its earlier reads are done, in order
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int x = lane + 64 * i;
        *(u32x4*)(mem + tile + 2 * place<DT>(x / kChunks, x % kChunks)) = vw[i];
      }
      own_lds_written();
      const int next = k0 + kPieceKeys;
      if (next < end) fetch(next);
      make_scores<kMode>(s[0], sc, slope, col.pos - k0);
      // past the piece's end are other pieces' keys
      softmax_step<DT, 1>(s, mul, k0 + 32 > min(wave_lo, key_hi), k0, min(col.lim, key_hi), m, l,
                          o);
      AddCols<T, DT, 1>(mem, tile, at_lane).run(s, o);
    }
    l = both_sum(l);
    __syncthreads();
    if (half == 0) {
      s_m[wave][lane] = m;
      s_l[wave][lane] = l;
    }
    leave_cols<DT>(s_raw, o);
    __syncthreads();
    // eight lanes a column join the four wavefronts, in order
    const int cc = threadIdx.x >> 3, e0 = (threadIdx.x & 7) * (DT / 8);
    const uint32_t c = col0 + cc;
    if (c < cols) {
      const Col w = column(a, d, hk, c, cols);
      float top = s_m[0][cc];
#pragma unroll
      for (int i = 1; i < 4; ++i) top = fmaxf(top, s_m[i][cc]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float f[4], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __builtin_amdgcn_exp2f(s_m[i][cc] - ref);
        sum = fmaf(f[i], s_l[i][cc], sum);
      }
      const int64_t row = d.qs + w.token;
      const int64_t at = ((int64_t)piece * a.heads_q + w.head) * a.docs.rows_q + row;
      const bool last = pieces == 1, none = w.lim <= 0;
      const float inv = none || sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int e = e0; e < e0 + DT / 8 && e < a.dim; e += 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[j] = fmaf(f[i], s_raw[(i * 32 + cc) * kStride + e + j], x[j]);
          if (last) x[j] = none ? 0.0f : x[j] * inv;
        }
        if (last)
          store_elems((T*)(a.out0 + row * a.out0_row + (int64_t)w.head * a.out0_head + e), x);
        else
          store_elems(a.part_o + at * a.dim + e, x);
      }
      if ((threadIdx.x & 7) == 0) {
        if (!last) {
          a.part_ml[at * 2] = top;
          a.part_ml[at * 2 + 1] = sum;
        } else if (a.lse) {
          a.lse[(int64_t)w.head * a.docs.rows_q + row] =
              none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        }
      }
    }
    if (a.col_units) break;  // the document's other tiles have workgroups
    __syncthreads();
  }
}

// The pieces of a column, joined in order: a workgroup a column; 16 groups of
// 16 lanes (8 elements a lane) take every 16th piece, and their sums are added
// in order.
template <typename T>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int tile_cols) {
  __shared__ float s_x[16][16][9], s_sum[16];
  int u = block_of(a) / tile_cols;
  const int hk = u % a.heads_k;
  u /= a.heads_k;
  const StepItem it = step_item(a, (a.pieces_last ? u : u * a.pieces) * a.heads_k);
  if (it.none) return;
  const Doc& d = it.d;
  const int pieces = pieces_of(a, d);
  if (pieces == 1) return;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const int sub = threadIdx.x & 15, group = threadIdx.x >> 4, e = sub * 8;
  const int64_t step = (int64_t)a.heads_q * a.docs.rows_q;
  for (uint32_t c = it.col0 + block_of(a) % tile_cols; c < cols; c += tile_cols) {
    const Col w = column(a, d, hk, c, cols);
    const int64_t row = d.qs + w.token, at = (int64_t)w.head * a.docs.rows_q + row;
    float top = -INFINITY;
    for (int i = threadIdx.x & 63; i < pieces; i += 64)
      top = fmaxf(top, a.part_ml[(at + i * step) * 2]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    for (int i = group; i < pieces; i += 16) {
      const f32x2 ml = *(const f32x2*)(a.part_ml + (at + i * step) * 2);
      const float f = __builtin_amdgcn_exp2f(ml.x - ref);
      sum = fmaf(f, ml.y, sum);
      if (e < a.dim) {
        float y[8];
        load_elems(a.part_o + (at + i * step) * a.dim + e, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(f, y[j], x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s_x[group][sub][j] = x[j];
    if (sub == 0) s_sum[group] = sum;
    __syncthreads();
    if (threadIdx.x < 16) {
      for (int g = 1; g < 16; ++g) {
        sum = g == 1 ? s_sum[0] + s_sum[1] : sum + s_sum[g];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += s_x[g][sub][j];
      }
      const bool none = w.lim <= 0;
      const float inv = none || sum == 0.0f ? 0.0f : 1.0f / sum;
      if (e < a.dim) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = none ? 0.0f : x[j] * inv;
        store_elems((T*)(a.out0 + row * a.out0_row + (int64_t)w.head * a.out0_head + e), x);
      }
      if (a.lse && e == 0)
        a.lse[at] = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
    if (a.col_units) break;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// p and ds of one 32 x 32 tile, in place of the products s and dp: register i
// has the logarithm lse(i), delta(i) and the bias away(i).
template <int kMode, typename Lse, typename Delta, typename Away>
__device__ inline void weigh(f32x16& s, f32x16& dp, const Scale& c, Lse lse, Delta delta,
                             Away away) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float f;
    const float x = score<kMode>(s[i], c, [&] { return away(i); }, f);
    const float p = __builtin_amdgcn_exp2f(kMode == 0 ? fmaf(x, c.mul, -lse(i)) : x - lse(i));
    float g = p * (dp[i] - delta(i));
    if constexpr (kMode & kCap) g *= f;
    s[i] = p;
    dp[i] = g;
  }
}

// The same where delta is still to be corrected (below): ds with the delta at
// hand, the derivative of a score's weight p f in place of p, and their sum's
// share sum_j p (dp - delta) over the keys below `room`.
template <int kMode, typename Away>
__device__ inline void weigh_once(f32x16& s, f32x16& dp, const Scale& c, float lse, float delta,
                                  Away away, bool part, int room, float& sum) {
  const int here = part ? room : 32;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float f;
    const float x = score<kMode>(s[i], c, [&] { return away(i); }, f);
    float p = __builtin_amdgcn_exp2f(x - lse);
    float g = p * (dp[i] - delta);
    if constexpr (kMode & kCap) {
      sum += result_row(i) < here ? g : 0.0f;
      p *= f;
      g *= f;
    }
    s[i] = p;
    dp[i] = g;
  }
  if (part) {
    const int last = only_here(room);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = result_row(i) < last ? s[i] : 0.0f;
      dp[i] = result_row(i) < last ? dp[i] : 0.0f;
    }
  }
  if constexpr (!(kMode & kCap)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += dp[i];
  }
}

// dq: the forward's loop, with p from the stored logarithm of the sum, and
// delta for the dk, dv kernel, which runs after it.  delta = do.o carries the
// roundings of o and of the weights that made it.  Where a row leans on few
// keys, so that o is as large as a value, they would be a third of the
// gradient's error.  Rows whose keys all stand in the first tile, and all rows
// under a distance bias, therefore take delta = sum_j p_j dp_j, the same number
// without those roundings, in a pass of its own over their keys.  Under a bias
// the pass can be spared where registers allow (here heads of 64 elements, all
// heads in the few-column form): with e = sum_j p_j (dp_j - delta), delta is
// corrected by e, and dq by -e sum_j p_j k_j, which is summed beside it.
// Causal documents of 3,360 and 13,024 tokens, 16 bf16 heads of 128 over 4,
// capped scores: 1.23 ms for three products a pair, 0.90 PFLOP/s.  By counters
// the vector unit issues in 72% of the cycles and the matrix unit works in 41%:
// bound by vector issue; the cap is as much vector work again as the exponential.
template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, 2) void attention_dq_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  // two buffers of a key and a value tile each
  constexpr int kTile = kKeys * DT * 2;
  __shared__ __align__(256) char mem[4 * kTile];
  const Lane<DT> at;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int hk = block_of(a) % a.heads_k;
  uint32_t local, units;
  Doc d;
  if (find_document<false>(a.docs, a.group, kCols, block_of(a) / a.heads_k, &local, &units, &d) < 0)
    return;
  const uint32_t col0 = (units - 1 - local) * kCols;
  const uint32_t cols = (uint32_t)d.ql * a.group;
  const Col col = column(a, d, hk, col0 + wave * 32 + (lane & 31), cols);
  const int64_t row = d.qs + col.token;
  const bool any = col.ok && col.lim > 0;
  V8 qf[DT / 16], df[DT / 16];
  load_cols<T, DT>(a.q + row * a.q_row + (int64_t)col.head * a.q_head, col.ok, a.dim, qf);
  load_cols<T, DT>(a.d + row * a.d_row + (int64_t)col.head * a.d_head, col.ok, a.dim, df);
  const int64_t place_of = (int64_t)col.head * a.docs.rows_q + row;
  const float lse = any ? a.lse[place_of] * kLog2e : INFINITY;
  float delta;
  {
    V8 of[DT / 16];
    load_cols<T, DT>(a.o + row * a.o_row + (int64_t)col.head * a.o_head, any, a.dim, of);
    delta = dot_cols<T, DT / 16>(of, df);
  }
  const float slope = (kMode & kGeneral) && a.slopes && col.ok ? a.slopes[col.head] * kLog2e
                                                               : 0.0f;
  const Scale sc = scale_of<kMode>(a);
  f32x16 g[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) g[i] = (f32x16)(0.0f);
  const int last_token = (int)((min(col0 + kCols, cols) - 1) / a.group);
  const int end = key_limit(a, d, last_token);
  const int wave_lo = __builtin_amdgcn_readlane(col.lim, 0);
  const int wave_hi = min(__builtin_amdgcn_readlane(col.lim, 31), end);
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  int buf = 0;
  auto copy = [&](int k0, int to) {
    copy_tile<DT, kKeys>(mem, to, kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
    copy_tile<DT, kKeys>(mem, to + kTile, vb + (int64_t)k0 * a.v_row, a.v_row, d.kl - k0, a.dim);
  };
  // the key tiles [0, last) in turn, each copied while the one before is used
  auto walk = [&](int last, auto use) {
    if (last <= 0) return;
    __syncthreads();
    copy(0, buf);
    for (int k0 = 0; k0 < last; k0 += kKeys, buf ^= 2 * kTile) {
      arrived();
      __syncthreads();
      if (k0 + kKeys < last) copy(k0 + kKeys, buf ^ (2 * kTile));
      if (k0 < wave_hi) use(k0);
    }
  };
  constexpr bool kOnce = DT == 64 && (kMode & kGeneral) != 0;
  const bool biased = (kMode & kGeneral) && a.slopes;
  const int block_lo = key_limit(a, d, (int)(col0 / a.group));
  if (!kOnce && (biased || block_lo <= kKeys)) {
    float sum = 0.0f;
    walk(biased ? end : min(end, kKeys), [&](int k0) {
#pragma unroll 1
      for (int r0 = 0; r0 < kKeys; r0 += 32) {
        f32x16 s, dp;
        const int rows = buf + r0 * DT * 2;
        two_products<T, DT>(mem, rows, rows + kTile, at, qf, df, s, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float f;
          const int at_key = k0 + r0 + result_row(i);
          const float x = score<kMode>(
              s[i], sc, [&] { return slope * fabsf((float)(col.pos - at_key)); }, f);
          const float p = __builtin_amdgcn_exp2f(kMode == 0 ? fmaf(x, sc.mul, -lse) : x - lse);
          sum = at_key < col.lim ? fmaf(p, dp[i], sum) : sum;
        }
      }
    });
    sum = both_sum(sum);
    if (biased || col.lim <= kKeys) delta = any ? sum : 0.0f;
  }
  if (!kOnce && col.ok && lane < 32) a.delta[place_of] = delta;
  f32x16 pk[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) pk[i] = (f32x16)(0.0f);
  float sum = 0.0f;
  walk(end, [&](int k0) {
#pragma unroll
    for (int r0 = 0; r0 < kKeys; r0 += 32) {
      f32x16 s, dp[1];
      const int rows = buf + r0 * DT * 2;
      two_products<T, DT>(mem, rows, rows + kTile, at, qf, df, s, dp[0]);
      AddCols<T, DT, 1> add(mem, rows, at);
      const int off = col.pos - k0 - r0;
      const auto away = [&](int i) { return slope * fabsf((float)(off - result_row(i))); };
      if constexpr (kOnce) {
        weigh_once<kMode>(s, dp[0], sc, lse, delta, away, k0 + kKeys > wave_lo,
                          col.lim - k0 - r0, sum);
        add.run(dp[0], g, s, pk);
        continue;
      }
      weigh<kMode>(s, dp[0], sc, [&](int) { return lse; }, [&](int) { return delta; }, away);
      if (k0 + kKeys > wave_lo) {
        const int room = only_here(col.lim - k0 - r0);
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[0][i] = result_row(i) < room ? dp[0][i] : 0.0f;
      }
      add.run(dp, g);
    }
  });
  if constexpr (kOnce) {
    sum = both_sum(sum);
    if (col.ok && lane < 32) a.delta[place_of] = any ? delta + sum : 0.0f;
#pragma unroll
    for (int i = 0; i < DT / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) g[i][j] = fmaf(-sum, pk[i][j], g[i][j]);
  }
  if (!col.ok) return;
  const bool none = col.lim <= 0;
  store_col<T, DT>(a.out0 + row * a.out0_row + (int64_t)col.head * a.out0_head, a.dim,
                   [&](int dt, int i) { return none ? 0.0f : g[dt][i] * a.scale; });
}

// dk and dv: a wavefront owns 32 keys of one key head, a workgroup 128, and
// walks the tokens that may see them, 32 at a time, for one query head after
// the other.  With a.parts a workgroup takes one query head of the group and
// leaves fp32 sums, which attention_heads_kernel adds over the group in order:
// with few keys there are otherwise too few workgroups to fill the chip.
// Heads of 128 elements keep the workgroup's values in LDS: beside both
// accumulators and the keys there is no room for them in registers.
// The same documents: 1.73 ms for four products a pair, 0.86 PFLOP/s, and 0.06
// for the sums over heads; two accumulators leave registers for two wavefronts a
// SIMD and for 32 columns, so every left operand is read from LDS for one
// product only (cycles with vector issue 53%, the matrix unit at work 37%, LDS
// 28%: two wavefronts do not cover each other's waits).
template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, 2) void attention_dkv_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  constexpr bool kValuesInLds = DT == 128;
  // two buffers of a tile of q and of do, then the values
  constexpr int kTile = kRows * DT * 2;
  __shared__ __align__(256) char mem[4 * kTile + (kValuesInLds ? kCols * DT * 2 : 0)];
  __shared__ __align__(16) float s_lse[2][kRows], s_delta[2][kRows];
  const Lane<DT> at;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int heads = a.parts ? a.heads_q : a.heads_k;
  const int hb = block_of(a) % heads;
  const int hk = a.parts ? hb / a.group : hb;
  const int head0 = a.parts ? hb : hb * a.group, nheads = a.parts ? 1 : a.group;
  uint32_t local, units;
  Doc d;
  if (find_document<true>(a.docs, 1, kCols, block_of(a) / heads, &local, &units, &d) < 0) return;
  const int key0 = (int)local * kCols;
  const int wkey = key0 + wave * 32;
  const int key = wkey + (lane & 31);
  const bool ok = key < d.kl;
  const int64_t row = d.ks + key;
  V8 kf[DT / 16], vf[kValuesInLds ? 1 : DT / 16];
  f32x16 gk[DT / 32], gv[DT / 32];
  load_cols<T, DT>(a.k + row * a.k_row + (int64_t)hk * a.k_head, ok, a.dim, kf);
  if constexpr (kValuesInLds) {
    copy_tile<DT, kCols>(mem, 4 * kTile,
                         a.v + (int64_t)(d.ks + key0) * a.v_row + (int64_t)hk * a.v_head, a.v_row,
                         d.kl - key0, a.dim);
  } else {
    load_cols<T, DT>(a.v + row * a.v_row + (int64_t)hk * a.v_head, ok, a.dim, vf);
  }
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) gk[i] = gv[i] = (f32x16)(0.0f);
  const Scale sc = scale_of<kMode>(a);
  // the first token that sees key0, and the tiles of a head
  const int shift = d.kl - d.ql;
  int first = 0;
  if (a.causal && key0 >= d.prefix) first = min(max(key0 - shift, 0), d.ql) / kRows * kRows;
  const int tiles = (d.ql - first + kRows - 1) / kRows;
  float r_lse = 0.0f, r_delta = 0.0f;
  // tokens t0 .. t0 + 31 of head head0 + h on their way into a buffer
  auto fetch = [&](int h, int t0, int buf) {
    const int64_t r = d.qs + t0;
    copy_tile<DT, kRows>(mem, buf * 2 * kTile,
                         a.q + r * a.q_row + (int64_t)(head0 + h) * a.q_head, a.q_row, d.ql - t0,
                         a.dim);
    copy_tile<DT, kRows>(mem, buf * 2 * kTile + kTile,
                         a.d + r * a.d_row + (int64_t)(head0 + h) * a.d_head, a.d_row, d.ql - t0,
                         a.dim);
    if (threadIdx.x < kRows) {
      const int t = t0 + (int)threadIdx.x;
      r_lse = INFINITY;
      r_delta = 0.0f;
      if (t < d.ql && key_limit(a, d, t) > 0) {
        const int64_t at = (int64_t)(head0 + h) * a.docs.rows_q + d.qs + t;
        r_lse = a.lse[at] * kLog2e;
        r_delta = a.delta[at];
      }
    }
  };
  auto put = [&](int buf) {
    if (threadIdx.x < kRows) {
      s_lse[buf][threadIdx.x] = r_lse;
      s_delta[buf][threadIdx.x] = r_delta;
    }
  };
  if (tiles > 0) {
    fetch(0, first, 0);
    put(0);
  }
  int buf = 0;
  for (int h = 0; h < nheads; ++h) {
    const float slope = (kMode & kGeneral) && a.slopes ? a.slopes[head0 + h] * kLog2e : 0.0f;
    for (int t0 = first; t0 < d.ql; t0 += kRows, buf ^= 1) {
      arrived();
      __syncthreads();
      const bool wrap = t0 + kRows >= d.ql, more = !wrap || h + 1 < nheads;
      if (more) fetch(wrap ? h + 1 : h, wrap ? first : t0 + kRows, buf ^ 1);
      // limits of the tile's rows grow with the token
      if (wkey < key_limit(a, d, t0 + kRows - 1)) {
        const int tile = buf * 2 * kTile;
        f32x16 s[1], dp[1];
        if constexpr (kValuesInLds)
          two_products_staged<T, DT, 2>(mem, tile, tile + kTile, 4 * kTile + wave * 32 * DT * 2, at,
                                     kf, s[0], dp[0]);
        else
          two_products<T, DT>(mem, tile, tile + kTile, at, kf, vf, s[0], dp[0]);
        const int off = t0 + shift - key;
        weigh<kMode>(s[0], dp[0], sc, [&](int i) { return s_lse[buf][result_row(i)]; },
                     [&](int i) { return s_delta[buf][result_row(i)]; },
                     [&](int i) { return slope * fabsf((float)(off + result_row(i))); });
        if (key_limit(a, d, t0) < wkey + 32) {
          const int here = only_here(key);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const bool seen = here < key_limit(a, d, t0 + result_row(i));
            s[0][i] = seen ? s[0][i] : 0.0f;
            dp[0][i] = seen ? dp[0][i] : 0.0f;
          }
        }
        AddCols<T, DT, 1, 2>(mem, tile + kTile, at).run(s, gv);
        AddCols<T, DT, 1, 2>(mem, tile, at).run(dp, gk);
      }
      if (more) put(buf ^ 1);
    }
  }
  arrived();  // the values, where no token sees these keys
  if (!ok) return;
  if (a.parts) {
    // [key row][query head][dk, dv][dim]
    float* p = a.part_o + (row * a.heads_q + hb) * 2 * a.dim;
#pragma unroll
    for (int dt = 0; dt < DT / 32; ++dt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = dt * 32 + 8 * i + 4 * (lane >> 5);
        if (e < a.dim) {
          const f32x4 x = {gk[dt][4 * i], gk[dt][4 * i + 1], gk[dt][4 * i + 2],
                           gk[dt][4 * i + 3]};
          const f32x4 y = {gv[dt][4 * i], gv[dt][4 * i + 1], gv[dt][4 * i + 2],
                           gv[dt][4 * i + 3]};
          *(f32x4*)(p + e) = x;
          *(f32x4*)(p + a.dim + e) = y;
        }
      }
    }
  } else {
    store_col<T, DT>(a.out0 + row * a.out0_row + (int64_t)hk * a.out0_head, a.dim,
                     [&](int dt, int i) { return gk[dt][i] * a.scale; });
    store_col<T, DT>(a.out1 + row * a.out1_row + (int64_t)hk * a.out1_head, a.dim,
                     [&](int dt, int i) { return gv[dt][i]; });
  }
}

// dq where there are few columns: as the forward's few-column form, a
// workgroup takes 32 columns, its wavefronts 32 keys each in turn, and their
// sums are added in order.  Six documents of 4,099 tokens in all, 8 fp16 heads of
// 64 over 2, a prefix and a bias: 32 us, bound by the longest document's walk
// (51 with a walk of its own for delta; 128-column form: 39).  Heads of 128
// under a bias: 80 (130).  They take one workgroup a compute unit, all registers:
// with two, 50 of them spill (three documents of 1,500 tokens 18 : 23 us).
template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, DT == 128 ? 1 : (kMode & kGeneral) ? 2 : 3) void
attention_dq_few_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  constexpr bool kOnce = (kMode & kGeneral) != 0;
  constexpr int kStride = DT + 4;
  __shared__ __align__(256) float s_raw[4 * 32 * kStride];
  __shared__ float s_delta[4][32];
  char* const mem = (char*)s_raw;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = wave * 32 * DT * 2;
  const Lane<DT> at;
  const int hk = block_of(a) % a.heads_k;
  uint32_t local, units;
  Doc d;
  if (find_document<false>(a.docs, a.group, 32, block_of(a) / a.heads_k, &local, &units, &d) < 0)
    return;
  const uint32_t col0 = (units - 1 - local) * 32, cols = (uint32_t)d.ql * a.group;
  const Col col = column(a, d, hk, col0 + (lane & 31), cols);
  const int64_t row = d.qs + col.token;
  const bool any = col.ok && col.lim > 0;
  V8 qf[DT / 16], df[DT / 16];
  load_cols<T, DT>(a.q + row * a.q_row + (int64_t)col.head * a.q_head, col.ok, a.dim, qf);
  load_cols<T, DT>(a.d + row * a.d_row + (int64_t)col.head * a.d_head, col.ok, a.dim, df);
  const int64_t place_of = (int64_t)col.head * a.docs.rows_q + row;
  const float lse = any ? a.lse[place_of] * kLog2e : INFINITY;
  float delta;
  {
    V8 of[DT / 16];
    load_cols<T, DT>(a.o + row * a.o_row + (int64_t)col.head * a.o_head, any, a.dim, of);
    delta = dot_cols<T, DT / 16>(of, df);
  }
  const float slope = (kMode & kGeneral) && a.slopes && col.ok ? a.slopes[col.head] * kLog2e
                                                               : 0.0f;
  const Scale sc = scale_of<kMode>(a);
  const int last_token = (int)((min(col0 + 32, cols) - 1) / a.group);
  const int end = key_limit(a, d, last_token);
  const int wave_lo = __builtin_amdgcn_readlane(col.lim, 0);
  const uint16_t* kb = a.k + (int64_t)d.ks * a.k_row + (int64_t)hk * a.k_head;
  const uint16_t* vb = a.v + (int64_t)d.ks * a.v_row + (int64_t)hk * a.v_head;
  Fragments<T, DT> kf, vf;
  auto fetch = [&](int k0) {
    kf.load(kb + (int64_t)k0 * a.k_row, a.k_row, d.kl - k0, a.dim);
    vf.load(vb + (int64_t)k0 * a.v_row, a.v_row, d.kl - k0, a.dim);
  };
  const bool biased = (kMode & kGeneral) && a.slopes;
  if (!kOnce && (biased || wave_lo <= kKeys)) {
    float sum = 0.0f;
    const int last = biased ? end : min(end, kKeys);
    int k0 = wave * 32;
    if (k0 < last) fetch(k0);
    for (; k0 < last; k0 += kPieceKeys) {
      const f32x16 s = kf.times(qf), dp = vf.times(df);
      if (k0 + kPieceKeys < last) fetch(k0 + kPieceKeys);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float f;
        const int key = k0 + result_row(i);
        const float x = score<kMode>(
            s[i], sc, [&] { return slope * fabsf((float)(col.pos - key)); }, f);
        const float p = __builtin_amdgcn_exp2f(kMode == 0 ? fmaf(x, sc.mul, -lse) : x - lse);
        sum = key < col.lim ? fmaf(p, dp[i], sum) : sum;
      }
    }
    sum = both_sum(sum);
    if (lane < 32) s_delta[wave][lane] = sum;
    __syncthreads();
    sum = ((s_delta[0][lane & 31] + s_delta[1][lane & 31]) + s_delta[2][lane & 31]) +
          s_delta[3][lane & 31];
    if (biased || col.lim <= kKeys) delta = any ? sum : 0.0f;
  }
  if (!kOnce && col.ok && wave == 0 && lane < 32) a.delta[place_of] = delta;
  f32x16 g[DT / 32], pk[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) g[i] = pk[i] = (f32x16)(0.0f);
  float sum = 0.0f;
  int k0 = wave * 32;
  if (k0 < end) fetch(k0);
  for (; k0 < end; k0 += kPieceKeys) {
    f32x16 s = kf.times(qf), dp[1] = {vf.times(df)};
    kf.store(mem, tile, at);
    own_lds_written();
    if (k0 + kPieceKeys < end) fetch(k0 + kPieceKeys);
    const int off = col.pos - k0;
    const auto away = [&](int i) { return slope * fabsf((float)(off - result_row(i))); };
    if constexpr (kOnce) {
      weigh_once<kMode>(s, dp[0], sc, lse, delta, away, k0 + 32 > wave_lo, col.lim - k0, sum);
      AddCols<T, DT, 1>(mem, tile, at).run(dp[0], g, s, pk);
      continue;
    }
    weigh<kMode>(s, dp[0], sc, [&](int) { return lse; }, [&](int) { return delta; }, away);
    if (k0 + 32 > wave_lo) {
      const int room = only_here(col.lim - k0);
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[0][i] = result_row(i) < room ? dp[0][i] : 0.0f;
    }
    AddCols<T, DT, 1>(mem, tile, at).run(dp, g);
  }
  if constexpr (kOnce) {
    sum = both_sum(sum);
    if (lane < 32) s_delta[wave][lane] = sum;
    __syncthreads();
    sum = ((s_delta[0][lane & 31] + s_delta[1][lane & 31]) + s_delta[2][lane & 31]) +
          s_delta[3][lane & 31];
    if (col.ok && wave == 0 && lane < 32) a.delta[place_of] = any ? delta + sum : 0.0f;
#pragma unroll
    for (int i = 0; i < DT / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) g[i][j] = fmaf(-sum, pk[i][j], g[i][j]);
  }
  __syncthreads();
  leave_cols<DT>(s_raw, g);
  __syncthreads();
  const int cc = threadIdx.x >> 3, e0 = (threadIdx.x & 7) * (DT / 8);
  if (col0 + cc >= cols) return;
  const Col w = column(a, d, hk, col0 + cc, cols);
  uint16_t* out = a.out0 + (int64_t)(d.qs + w.token) * a.out0_row + (int64_t)w.head * a.out0_head;
  for (int e = e0; e < e0 + DT / 8 && e < a.dim; e += 8) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* p = s_raw + cc * kStride + e + j;
      x[j] = ((p[0] + p[32 * kStride]) + p[64 * kStride]) + p[96 * kStride];
      x[j] = w.lim <= 0 ? 0.0f : x[j] * a.scale;
    }
    store_elems((T*)(out + e), x);
  }
}

// dk and dv where there are few keys: a workgroup takes 32 keys of a key head,
// its wavefronts 32 tokens of a query head each in turn, and their sums are
// added in order (a.parts: as above).  The same documents: 42 us, bound as above.
template <typename T, int DT, int kMode>
__global__ __launch_bounds__(256, DT == 128 ? 1 : 2) void attention_dkv_few_kernel(AttnArgs a) {
  typedef typename Mat<T>::V8 V8;
  constexpr int kStride = DT + 4;
  constexpr int kTile = 32 * DT * 2;
  constexpr int kBytes = 8 * kTile > 4 * 32 * kStride * 4 ? 8 * kTile : 4 * 32 * kStride * 4;
  __shared__ __align__(256) float s_raw[kBytes / 4];
  __shared__ __align__(16) float s_row[4][2][32];
  char* const mem = (char*)s_raw;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = wave * 2 * kTile;
  const Lane<DT> at;
  const int heads = a.parts ? a.heads_q : a.heads_k;
  const int hb = block_of(a) % heads;
  const int hk = a.parts ? hb / a.group : hb;
  const int head0 = a.parts ? hb : hb * a.group, nheads = a.parts ? 1 : a.group;
  uint32_t local, units;
  Doc d;
  if (find_document<true>(a.docs, 1, 32, block_of(a) / heads, &local, &units, &d) < 0) return;
  const int key0 = (int)local * 32, key = key0 + (lane & 31);
  const int64_t row = d.ks + key0;
  Fragments<T, DT> kf, vf, qf, df;
  kf.load(a.k + row * a.k_row + (int64_t)hk * a.k_head, a.k_row, d.kl - key0, a.dim);
  vf.load(a.v + row * a.v_row + (int64_t)hk * a.v_head, a.v_row, d.kl - key0, a.dim);
  f32x16 gk[DT / 32], gv[DT / 32];
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) gk[i] = gv[i] = (f32x16)(0.0f);
  const Scale sc = scale_of<kMode>(a);
  const int shift = d.kl - d.ql;
  int first = 0;
  if (a.causal && key0 >= d.prefix) first = min(max(key0 - shift, 0), d.ql) / 32 * 32;
  const int tiles = (d.ql - first + 31) / 32, total = tiles * nheads;
  float r_lse = 0.0f, r_delta = 0.0f;
  // tile n: tokens first + 32 (n % tiles) of query head head0 + n / tiles
  auto fetch = [&](int n) {
    const int h = n / tiles, t0 = first + (n - h * tiles) * 32, head = head0 + h;
    const int64_t r = d.qs + t0;
    qf.load(a.q + r * a.q_row + (int64_t)head * a.q_head, a.q_row, d.ql - t0, a.dim);
    df.load(a.d + r * a.d_row + (int64_t)head * a.d_head, a.d_row, d.ql - t0, a.dim);
    const int t = t0 + (lane & 31);
    r_lse = INFINITY;
    r_delta = 0.0f;
    if (t < d.ql && key_limit(a, d, t) > 0) {
      const int64_t p = (int64_t)head * a.docs.rows_q + d.qs + t;
      r_lse = a.lse[p] * kLog2e;
      r_delta = a.delta[p];
    }
  };
  int n = wave;
  if (n < total) fetch(n);
  for (; n < total; n += 4) {
    const int h = n / tiles, t0 = first + (n - h * tiles) * 32;
    f32x16 s[1] = {qf.times(kf.f)}, dp[1] = {df.times(vf.f)};
    qf.store(mem, tile, at);
    df.store(mem, tile + kTile, at);
    if (lane < 32) {
      s_row[wave][0][lane] = r_lse;
      s_row[wave][1][lane] = r_delta;
    }
    own_lds_written();
    if (n + 4 < total) fetch(n + 4);
    const float slope =
        (kMode & kGeneral) && a.slopes ? a.slopes[head0 + h] * kLog2e : 0.0f;
    const int off = t0 + shift - key;
    weigh<kMode>(s[0], dp[0], sc, [&](int i) { return s_row[wave][0][result_row(i)]; },
                 [&](int i) { return s_row[wave][1][result_row(i)]; },
                 [&](int i) { return slope * fabsf((float)(off + result_row(i))); });
    if (key_limit(a, d, t0) < key0 + 32) {
      const int here = only_here(key);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool seen = here < key_limit(a, d, t0 + result_row(i));
        s[0][i] = seen ? s[0][i] : 0.0f;
        dp[0][i] = seen ? dp[0][i] : 0.0f;
      }
    }
    AddCols<T, DT, 1>(mem, tile + kTile, at).run(s, gv);
    AddCols<T, DT, 1>(mem, tile, at).run(dp, gk);
  }
  const int cc = threadIdx.x >> 3, e0 = (threadIdx.x & 7) * (DT / 8);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    __syncthreads();
    leave_cols<DT>(s_raw, w ? gv : gk);
    __syncthreads();
    if (key0 + cc >= d.kl) continue;
    uint16_t* out = w ? a.out1 + (row + cc) * a.out1_row + (int64_t)hk * a.out1_head
                      : a.out0 + (row + cc) * a.out0_row + (int64_t)hk * a.out0_head;
    for (int e = e0; e < e0 + DT / 8 && e < a.dim; e += 8) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* p = s_raw + cc * kStride + e + j;
        x[j] = ((p[0] + p[32 * kStride]) + p[64 * kStride]) + p[96 * kStride];
        if (!w && !a.parts) x[j] *= a.scale;
      }
      if (a.parts)
        store_elems(a.part_o + (((row + cc) * a.heads_q + hb) * 2 + w) * a.dim + e, x);
      else
        store_elems((T*)(out + e), x);
    }
  }
}

// Sums of a key head's dk and dv over its query heads, in order: 16 keys a
// workgroup, 16 lanes a key, 8 elements a lane.
template <typename T>
__global__ __launch_bounds__(256) void attention_heads_kernel(AttnArgs a) {
  const int hk = block_of(a) % a.heads_k;
  uint32_t local, units;
  Doc d;
  if (find_document<true>(a.docs, 1, 16, block_of(a) / a.heads_k, &local, &units, &d) < 0) return;
  const int e = (threadIdx.x & 15) * 8, key = (int)local * 16 + (threadIdx.x >> 4);
  if (e >= a.dim || key >= d.kl) return;
  const int64_t row = d.ks + key;
  float x[8], y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
  const float* p = a.part_o + (row * a.heads_q + (int64_t)hk * a.group) * 2 * a.dim + e;
#pragma unroll 4
  for (int h = 0; h < a.group; ++h) {
    float u[8], w[8];
    load_elems(p + (int64_t)h * 2 * a.dim, u);
    load_elems(p + ((int64_t)h * 2 + 1) * a.dim, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] += u[j];
      y[j] += w[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] *= a.scale;
  store_elems((T*)(a.out0 + row * a.out0_row + (int64_t)hk * a.out0_head + e), x);
  store_elems((T*)(a.out1 + row * a.out1_row + (int64_t)hk * a.out1_head + e), y);
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

// Whether `blocks` workgroups of the 128-column form are too few: with less
// than one a compute unit, its time is its longest document's, which the
// few-column form divides by four at half the throughput.  Under a distance
// bias a key takes longer (and dq's 128-column form walks the keys of
// 128-element heads twice), and the turning point is later.  Measured, us,
// 128-column form : few-column form (forward; dq), heads of 64:
//   74 workgroups  7.4 : 6.5;  8.8 : 8.3      262  16.6 : 19.7;  17.7 : 26.0
//   268 with a bias and uneven documents      36.7 : 25.2;  39 : 32
bool few_columns(const gs_attention_config& cfg, int64_t blocks) {
  return blocks < (cfg.slopes ? 512 : 256);
}

// The few-column form, and how many pieces it cuts a document's keys into.
struct Split {
  bool few, col_units, pieces_last;
  int pieces, piece;
  int64_t units;  // column tiles of a key head
  int cols;       // columns of a tile that a document may have
};
Split split_of(const gs_attention_config& cfg, const gs_documents& d, int64_t rows_q,
               int64_t rows_k) {
  Split o = {};
  const int64_t group = cfg.heads_q / cfg.heads_k;
  const int64_t longest_q = d.max_q_len > 0 && d.max_q_len < rows_q ? d.max_q_len : rows_q;
  const int64_t longest_k = d.max_k_len > 0 && d.max_k_len < rows_k ? d.max_k_len : rows_k;
  // one tile a document, or a look-up
  o.col_units = longest_q * group > 32;
  o.units = o.col_units ? unit_bound(rows_q * group, 32, d.count) : d.count;
  o.cols = o.col_units ? 32 : (int)(longest_q * group);
  o.few = !o.col_units ||
          few_columns(cfg, unit_bound(rows_q * group, kCols, d.count) * cfg.heads_k);
  const int64_t base = o.units * cfg.heads_k;
  // Workgroups wanted: with few documents a round of what the chip holds (four
  // caches of 120,001 keys in all, us: 77, 63, 78, 70, 72 at 512, 768, 1024,
  // 1536, 2048); with many of uneven length more, so that the long ones end
  // sooner (64 caches of 100,003: 87, 85, 75, 78, 72 at 512, 768, 1536, 2048,
  // 3072).  Column tiles that are looked up are many already.  Even caches do
  // not care (8 to 64 caches of eight heads of 64, 100,000 keys: 42 to 44 at any
  // of these); of the uneven ones, those with just under 256 tiles lose by the
  // step (31 caches: 69 at 768, 47 at 3072; 32 caches: 66, 45).
  o.pieces_last = base >= 256;
  const int64_t target = o.col_units ? 512 : o.pieces_last ? 3072 : 768;
  const int64_t want = (target + base - 1) / base;
  int64_t piece = (longest_k + want - 1) / want;
  piece = (piece + kPieceKeys - 1) / kPieceKeys * kPieceKeys;
  const int64_t least = o.col_units ? 8 * kPieceKeys : 2 * kPieceKeys;
  if (piece < least) piece = least;
  // the join of thousands of columns costs 12 us or so (one piece : several, us:
  // documents of 1,500 tokens 14 : 28, of 2,500 37 : 37, of 4,000 51 : 40)
  if (o.col_units && longest_k <= 20 * kPieceKeys) piece = 20 * kPieceKeys;
  if (piece > (1 << 30)) piece = 1 << 30;
  o.piece = (int)piece;
  o.pieces = (int)((longest_k + piece - 1) / piece);
  if (o.pieces < 1) o.pieces = 1;
  return o;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The few-key form of dk and dv: few workgroups of the 128-key form even with
// one to a query head.  Heads of 128 elements fill a SIMD's registers with one
// wavefront there, and turn earlier.  128-key form : few-key form, us: heads of
// 64, 304 workgroups 33 : 31 (under a bias, uneven documents, 63 : 42); heads
// of 128, 64 workgroups 93 : 52; training passes with 114 137 : 96, with 228
// 167 : 153, with 304 160 : 170.
bool few_keys(const gs_attention_config& cfg, int64_t rows_k, int32_t count) {
  return unit_bound(rows_k, kCols, count) * cfg.heads_q < (cfg.head_dim > 64 ? 256 : 384);
}

// Whether dk and dv are summed per query head first: there are otherwise few
// workgroups, whose walks over all heads of a group end late.  Backward of
// documents of 2,048 tokens, us, per key head : per query head and summed, by
// the workgroups of the former:
//   16 heads of 128 over 4:  136  450 : 227;  544  729 : 653;  1,632  2056 : 1826;
//                            2,176  2567 : 2412;  3,264  3796 : 3716
//   16 heads of 64 over 8:   2,176  734 : 750;  4,352  1371 : 1434
bool head_parts(const gs_attention_config& cfg, const gs_documents& d, int64_t rows_k) {
  if (cfg.heads_q == cfg.heads_k) return false;
  const int step = few_keys(cfg, rows_k, d.count) ? 32 : kCols;
  return unit_bound(rows_k, step, d.count) * cfg.heads_k < 2048;
}

// The kernels of one element type, head size and way to make scores.
template <typename T, int DT, int kMode>
struct Run {
  // kernel<<<blocks, 256>>>(a, more ...)
  template <typename K, typename... More>
  static hipError_t launch(K kernel, int64_t blocks, AttnArgs a, hipStream_t s, More... more) {
    return launch_all(blocks, 256, [&](uint32_t first, dim3 grid) {
      a.block0 = first;
      kernel<<<grid, dim3(256), 0, s>>>(a, more...);
    });
  }

  static hipError_t fwd(const AttnArgs& a, const Split& p, hipStream_t s) {
    if (p.few) {
      const int64_t tiles = p.units * a.heads_k;
      const hipError_t e =
          launch(attention_step_kernel<T, DT, kMode>, tiles * a.pieces, a, s);
      if (e != hipSuccess || a.pieces == 1) return e;
      return launch(attention_join_kernel<T>, tiles * p.cols, a, s, p.cols);
    }
    const int64_t columns = (int64_t)a.docs.rows_q * a.group;
    return launch(attention_fwd_kernel<T, DT, kMode>,
                  unit_bound(columns, kCols, a.docs.count) * a.heads_k, a, s);
  }

  static hipError_t bwd(AttnArgs a, const gs_attention_config& cfg, const gs_heads& dq,
                        const gs_heads& dk, const gs_heads& dv, hipStream_t s) {
    hipError_t e;
    if (a.docs.rows_q > 0) {
      a.out0 = (uint16_t*)dq.data; a.out0_row = dq.row; a.out0_head = dq.head;
      const int64_t columns = (int64_t)a.docs.rows_q * a.group;
      const int64_t blocks = unit_bound(columns, kCols, a.docs.count) * a.heads_k;
      if (few_columns(cfg, blocks))
        e = launch(attention_dq_few_kernel<T, DT, kMode>,
                   unit_bound(columns, 32, a.docs.count) * a.heads_k, a, s);
      else
        e = launch(attention_dq_kernel<T, DT, kMode>, blocks, a, s);
      if (e != hipSuccess) return e;
    }
    a.out0 = (uint16_t*)dk.data; a.out0_row = dk.row; a.out0_head = dk.head;
    a.out1 = (uint16_t*)dv.data; a.out1_row = dv.row; a.out1_head = dv.head;
    const int heads = a.parts ? a.heads_q : a.heads_k;
    if (few_keys(cfg, a.docs.rows_k, a.docs.count))
      e = launch(attention_dkv_few_kernel<T, DT, kMode>,
                 unit_bound(a.docs.rows_k, 32, a.docs.count) * heads, a, s);
    else
      e = launch(attention_dkv_kernel<T, DT, kMode>,
                 unit_bound(a.docs.rows_k, kCols, a.docs.count) * heads, a, s);
    if (e != hipSuccess || !a.parts) return e;
    return launch(attention_heads_kernel<T>,
                  unit_bound(a.docs.rows_k, 16, a.docs.count) * a.heads_k, a, s);
  }
};

template <typename T, int DT, typename F>
hipError_t with_mode(const AttnArgs& a, F f) {
  const bool cap = a.softcap > 0.0f, general = a.slopes != nullptr || !(a.scale > 0.0f);
  // (one kind of scores serves all wide caps, which are rare)
  if (a.softcap > kWideCap) return f(Run<T, DT, kCap | kGeneral | kWide>());
  if (cap) return general ? f(Run<T, DT, kCap | kGeneral>()) : f(Run<T, DT, kCap>());
  return general ? f(Run<T, DT, kGeneral>()) : f(Run<T, DT, 0>());
}

// Heads of up to 64 elements, or of up to 128 (shorter ones are filled with
// zeros in LDS).
template <typename F>
hipError_t dispatch(const gs_attention_config& cfg, const AttnArgs& a, F f) {
  if (cfg.dtype == GS_BF16)
    return cfg.head_dim > 64 ? with_mode<Bf16, 128>(a, f) : with_mode<Bf16, 64>(a, f);
  return cfg.head_dim > 64 ? with_mode<F16, 128>(a, f) : with_mode<F16, 64>(a, f);
}

}  // namespace

extern "C" {

// Whether the forward's workgroups search the documents for their tokens.
bool gs_attention_searches(const gs_attention_config& cfg, const gs_documents& d,
                           int64_t rows_q) {
  return split_of(cfg, d, rows_q, 0).col_units;
}

size_t gs_attention_fwd_bytes(const gs_attention_config& cfg, const gs_documents& d,
                              int64_t rows_q, int64_t rows_k) {
  if (d.count == 0 || rows_q == 0) return 0;
  const Split p = split_of(cfg, d, rows_q, rows_k);
  if (!p.few || p.pieces == 1) return 0;
  const size_t columns = (size_t)p.pieces * cfg.heads_q * rows_q;
  return align256(columns * 2 * sizeof(float)) + columns * cfg.head_dim * sizeof(float);
}

size_t gs_attention_bwd_bytes(const gs_attention_config& cfg, const gs_documents& d,
                              int64_t rows_q, int64_t rows_k) {
  if (d.count == 0) return 0;
  size_t n = align256((size_t)rows_q * cfg.heads_q * sizeof(float));
  if (head_parts(cfg, d, rows_k))
    n += (size_t)rows_k * cfg.heads_q * 2 * cfg.head_dim * sizeof(float);
  return n;
}

hipError_t gs_launch_attention_fwd(const gs_attention_config& cfg, const gs_documents& d,
                                   int64_t rows_q, int64_t rows_k, const gs_heads& q,
                                   const gs_heads& k, const gs_heads& v, const gs_heads& out,
                                   float* lse, void* workspace, hipStream_t s) {
  AttnArgs a = make_args(cfg, d, rows_q, rows_k, q, k, v);
  a.out0 = (uint16_t*)out.data; a.out0_row = out.row; a.out0_head = out.head;
  a.lse = lse;
  const Split p = split_of(cfg, d, rows_q, rows_k);
  a.pieces = p.pieces;
  a.piece = p.piece;
  a.col_units = p.col_units;
  a.tiles = (int)p.units;
  a.pieces_last = p.pieces_last;
  a.part_ml = (float*)workspace;
  a.part_o = (float*)((char*)workspace +
                      align256((size_t)p.pieces * cfg.heads_q * rows_q * 2 * sizeof(float)));
  return dispatch(cfg, a, [&](auto run) { return run.fwd(a, p, s); });
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
  a.part_o = (float*)((char*)workspace + align256((size_t)rows_q * cfg.heads_q * sizeof(float)));
  a.parts = head_parts(cfg, d, rows_k);
  return dispatch(cfg, a, [&](auto run) { return run.bwd(a, cfg, dq, dk, dv, s); });
}

}  // extern "C"
