// linear8.hip — rows brought to 8 bits, and products of them with 8-bit
// weights.
//
//   scale_i = max_k |x_ik| / 127,  u_ik = rint(127 x_ik / max),
//   y_ij = (sum_k u_ik w_jk) (scale_i wscale_j) + bias_j.
//
// The sums are whole numbers in 32 bits, so no order of them changes a result.
// Codes are formed in 64 bits: the fp32 product would put a value next to the
// border of two codes into either.
//
// What bounds it.  Few rows: reading the weights, and one launch or two.  Many: the
// matrix unit, at work in 56% of the cycles, at 1.7 to 1.9 GHz under this load (16,384 rows
// of 4,096 by 8,192 in 550 to 562 us, 2.0 POP/s, 50 us of it the codes; the products
// alone, without loads or results, take 445).
//
// The figures beside the rules below: bf16 with a bias, calls captured in a graph
// over weights and rows of 600 MB that take turns, so that none come from a cache.
#include "tokens.h"

namespace gs {

struct LinearArgs {
  int64_t rows;
  int inputs, outputs;
  const void* x;         // kOwn: rows as they came
  int64_t x_row;
  const int8_t* u;       // [rows][inputs]
  const float* u_scale;  // [rows]
  const int8_t* w;       // [outputs][inputs]
  const float* w_scale;  // [outputs]
  const float* bias;     // [outputs] or NULL
  void* y;
  int64_t y_row;
  uint32_t tiles_n;  // tiles over the outputs
  uint32_t tiles;
};

// What a row's largest magnitude makes of it.  A row with an infinity or a NaN
// has no codes: its scale is NaN, and so is all that comes of it.
struct RowScale {
  float scale;
  double inv;
  __device__ inline explicit RowScale(float top) {
    const bool none = top < kLeastSpan, wrong = !(top < __builtin_huge_valf());
    inv = none || wrong ? 0.0 : 127.0 / (double)top;
    scale = wrong ? __builtin_nanf("") : none ? 0.0f : (float)((double)top / 127.0);
  }
};

// Eight codes.
__device__ inline u32x2 codes_of(const float (&v)[8], const RowScale& r) {
  uint32_t w[2] = {0, 0};
  if (r.scale == r.scale) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= (uint32_t)(code_of(v[i], r.inv) & 255) << (8 * (i & 3));
  }
  return u32x2{w[0], w[1]};
}

// kLanes lanes a row; each keeps up to kKeep pieces of eight elements in
// registers between the maximum and the codes and reads the others again.  Memory
// bound: 16,384 rows of 4,096 in bf16 in 50 us (201 MB, 4.0 TB/s); small ones a launch.
template <typename T, int kLanes>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int64_t rows, int channels, const T* x,
                                                            int64_t x_row, int8_t* codes,
                                                            float* scales, uint32_t block0) {
  constexpr int kKeep = 4;
  __shared__ float s_top[4];
  const int64_t row = (int64_t)(block0 + blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes;
  const int at = (threadIdx.x % kLanes) * 8;
  const bool here = row < rows;
  const T* in = x + (here ? row : 0) * x_row;
  float kept[kKeep][8];
  float top = 0.0f;
  bool bad = false;
  auto look = [&](const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(v[i]));
      bad = bad || !(fabsf(v[i]) < __builtin_huge_valf());
    }
  };
#pragma unroll
  for (int p = 0; p < kKeep; ++p) {
    const int e = at + p * kLanes * 8;
    if (here && e < channels) {
      load_elems(in + e, kept[p]);
      look(kept[p]);
    }
  }
  for (int e = at + kKeep * kLanes * 8; here && e < channels; e += kLanes * 8) {
    float v[8];
    load_elems(in + e, v);
    look(v);
  }
  if (bad) top = __builtin_huge_valf();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if constexpr (kLanes == 256) {
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  }
  if (!here) return;
  const RowScale r(top);
  if (threadIdx.x % kLanes == 0) scales[row] = r.scale;
  int8_t* out = codes + row * channels;
#pragma unroll
  for (int p = 0; p < kKeep; ++p) {
    const int e = at + p * kLanes * 8;
    if (e < channels) *(u32x2*)(out + e) = codes_of(kept[p], r);
  }
  for (int e = at + kKeep * kLanes * 8; e < channels; e += kLanes * 8) {
    float v[8];
    load_elems(in + e, v);
    *(u32x2*)(out + e) = codes_of(v, r);
  }
}

// Up to 16 rows: the product is the reading of the weights.  A workgroup has 16
// outputs, its wavefronts a share of the inputs each; weights and codes go from
// memory straight into the operands of the 16x16x64 instruction (rows lane %
// 16, 16 inputs a lane), and the wavefronts' sums meet in LDS.  Weights of
// the first kAheadOfAll steps are on their way before anything else is looked at:
// 16.8 MB of them, one row of 2,048 by 8,192, take 7.1 us (2.4 TB/s; a launch alone
// is about 3), 6.2 where a few such calls take turns.
// 16 wavefronts where there is a workgroup a compute unit or less, 8 where there
// are more (us, 16 : 8; one row of 4,096 by 4,096 7.4 : 7.6, of 2,048 by 8,192
// 9.5 : 7.1).
//
// kOwn: rows are brought to codes here, by every workgroup for itself while its
// weights are on their way, which saves a launch: up to eight rows of at most
// kOwnElems elements (rows rounded up to a power of two).
constexpr int kAheadOfAll = 64;
constexpr int kUnits = 256;  // compute units
constexpr int kOutputsOf16 = 16 * kUnits;
constexpr int kKeep = 4;  // pieces of eight elements, a lane
template <int kWaves>
constexpr int kOwnElems = kWaves * 64 * 8 * kKeep;
template <typename T, int kWaves, bool kOwn>
__global__ void __launch_bounds__(kWaves * 64, 4) linear_few_kernel(LinearArgs a) {
  constexpr int kAhead = kAheadOfAll / kWaves;
  __shared__ i32x4 s_sum[kWaves][64];
  __shared__ uint32_t s_top[8];
  // a row of codes is 16 bytes longer than its inputs, so that the 16 rows read
  // together fall on different banks
  __shared__ __align__(16) int8_t s_codes[kOwn ? kOwnElems<kWaves> + 8 * 16 : 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16;
  const int steps = (a.inputs + 63) / 64;
  const int share = (steps + kWaves - 1) / kWaves;
  const int first = wave * share, last = min(steps, first + share);
  const int part = 16 * (lane >> 4);
  // rows past the end repeat the last one; what comes of them is not stored
  const int8_t* w = a.w + (int64_t)min(n0 + (lane & 15), a.outputs - 1) * a.inputs + part;
  i32x4 ahead[kAhead];
  auto load_weights = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      ahead[i] = i32x4{0, 0, 0, 0};
      if (s0 + i < last && 64 * (s0 + i) + part < a.inputs)  // inputs are a multiple of 16
        ahead[i] = *(const i32x4*)(w + 64 * (s0 + i));
    }
  };
  load_weights(first);
  if constexpr (kOwn) {
    // up to eight rows: an eighth of the wavefronts a row, or more
    const int rows = (int)a.rows, each = kWaves / (rows <= 2 ? rows : rows <= 4 ? 4 : 8);
    const int row = wave / each, at = ((wave % each) * 64 + lane) * 8;
    const bool mine = row < rows;
    const T* x = (const T*)a.x + (mine ? row : 0) * a.x_row;
    if (threadIdx.x < 8) s_top[threadIdx.x] = 0;
    float kept[kKeep][8];
#pragma unroll
    for (int p = 0; p < kKeep; ++p) {
      const int e = at + p * each * 512;
      if (mine && e < a.inputs) load_elems(x + e, kept[p]);
    }
    __syncthreads();
    // the largest magnitude as a whole number: an infinity or a NaN is above all
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < kKeep; ++p) {
      if (!mine || at + p * each * 512 >= a.inputs) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, __builtin_bit_cast(uint32_t, kept[p][i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if (mine && lane == 0) atomicMax(&s_top[row], top);
    __syncthreads();
    if (mine) {
      const RowScale r(__builtin_bit_cast(float, s_top[row]));
#pragma unroll
      for (int p = 0; p < kKeep; ++p) {
        const int e = at + p * each * 512;
        if (e < a.inputs) *(u32x2*)(s_codes + row * (a.inputs + 16) + e) = codes_of(kept[p], r);
      }
    }
    __syncthreads();
  }
  // the results that this lane will store: one row, four outputs
  const int rows = (int)a.rows, m = lane & 15, n = n0 + 4 * (lane >> 4);
  const int8_t* u = kOwn ? s_codes + min(m, rows - 1) * (a.inputs + 16) + part
                         : a.u + (int64_t)min(m, rows - 1) * a.inputs + part;
  const bool stored = wave == 0 && m < rows && n < a.outputs;
  float scale = 0.0f, w_scale[4] = {0.0f, 0.0f, 0.0f, 0.0f}, bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (stored) {
    if (!kOwn) scale = a.u_scale[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w_scale[i] = a.w_scale[n + i];
      if (a.bias) bias[i] = a.bias[n + i];
    }
  }
  i32x4 sum = {0, 0, 0, 0};
  for (int s0 = first; s0 < last; s0 += kAhead) {
    if (s0 > first) load_weights(s0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      i32x4 y = {0, 0, 0, 0};
      if (s0 + i < last && 64 * (s0 + i) + part < a.inputs) y = *(const i32x4*)(u + 64 * (s0 + i));
      sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(ahead[i], y, sum, 0, 0, 0);
    }
  }
  s_sum[wave][lane] = sum;
  __syncthreads();
  if (!stored) return;
#pragma unroll
  for (int i = 1; i < kWaves; ++i) sum += s_sum[i][lane];
  if (kOwn) scale = RowScale(__builtin_bit_cast(float, s_top[m & 7])).scale;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (float)sum[i] * (scale * w_scale[i]);
    if (a.bias) v[i] += bias[i];
  }
  store_elems((T*)a.y + (int64_t)m * a.y_row + n, v);
}

// Place in a staged tile of 128-byte rows: 16-byte chunk c of row r stands at
// chunk c ^ turn(r).  Outputs are read in the order 0..3, 16..19, 4..7, 20..23
// ..., rows in their own: of sixteen rows read together the eight even ones have
// eight different turns, and so have the odd ones, whose chunks stand in the other
// half of the 64 banks.
template <bool kOutputs>
__device__ inline int turn(int r) {
  return kOutputs ? ((r >> 1) & 3) | ((r >> 2) & 4) : (r >> 1) & 7;
}

// Copies kRows rows of 128 bytes from column k on into LDS, without passing
// through registers.  at: each lane's source offsets, of row and chunk.
template <int kRows, int kWaves, bool kOutputs>
struct Stage {
  static constexpr int kCopies = kRows / 8 / kWaves;
  uint32_t at[kCopies];
  int chunk[kCopies];
  __device__ inline void start(int inputs) {
    const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) % kWaves;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int r = (i * kWaves + wave) * 8 + (lane >> 3);
      chunk[i] = ((lane & 7) ^ turn<kOutputs>(r)) * 16;
      at[i] = (uint32_t)(r * inputs + chunk[i]);
    }
  }
  __device__ inline void copy(const i32x4& rsrc, uint32_t lds, int k, int inputs) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % kWaves);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      // chunks past the row's end arrive as zeros
      const uint32_t from = k + chunk[i] < inputs ? at[i] + (uint32_t)k : 0x80000000u;
      const uint32_t to = lds + (i * kWaves + wave) * 1024;
      asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(
                       from),
                   "s"(rsrc), "s"(to)
                   : "memory", "m0");
    }
  }
};

__device__ inline i32x4 rows_from(const int8_t* base, int64_t bytes) {
  const uint64_t address = (uint64_t)base;
  return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)address),
               (int)__builtin_amdgcn_readfirstlane((uint32_t)(address >> 32) & 0xffff),
               (int)__builtin_amdgcn_readfirstlane((uint32_t)bytes), 0x00027000};
}

// More rows: tiles of kM rows by kN outputs, kWm by kWn wavefronts of 32x32x32
// products, 128 inputs a step, kStages of them in LDS: while one is multiplied the
// next ones are copied in.  With kSplit above 1 that many such groups of wavefronts
// take the steps in turn, each with stages of its own, and their sums meet at the end.
template <typename T, int kM, int kN, int kWm, int kWn, int kStages, int kSplit>
__global__ void __launch_bounds__(kWm* kWn* kSplit * 64) linear_many_kernel(LinearArgs a) {
  constexpr int kWaves = kWm * kWn;
  constexpr int kTm = kM / kWm / 32, kTn = kN / kWn / 32;
  constexpr int kBytes = (kM + kN) * 128;
  constexpr int kCopies = (kM + kN) / 8 / kWaves;  // of a stage, a wavefront
  __shared__ __align__(1024) char s_mem[kSplit * kStages * kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % kWaves);
  const int group = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / kWaves);
  // Workgroups go to the eight XCDs in turn; each XCD takes a run of tiles, in
  // blocks of eight tiles of rows, so that its L2 holds what they share.
  const uint32_t each = (a.tiles + 7) / 8;
  const uint32_t tile = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= each || tile >= a.tiles) return;
  const uint32_t tiles_m = a.tiles / a.tiles_n, block = tile / (8 * a.tiles_n);
  const uint32_t tall = min(8u, tiles_m - block * 8);
  const uint32_t in_block = tile - block * 8 * a.tiles_n;
  const int64_t m0 = (int64_t)(block * 8 + in_block % tall) * kM;
  const int n0 = (int)(in_block / tall) * kN;
  const int64_t rows = min(a.rows - m0, (int64_t)kM);
  const int outputs = min(a.outputs - n0, kN);
  const i32x4 from_u = rows_from(a.u + m0 * a.inputs, rows * a.inputs);
  const i32x4 from_w = rows_from(a.w + (int64_t)n0 * a.inputs, (int64_t)outputs * a.inputs);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)s_mem;
  Stage<kM, kWaves, false> stage_u;
  Stage<kN, kWaves, true> stage_w;
  stage_u.start(a.inputs);
  stage_w.start(a.inputs);
  auto copy = [&](int s, int buffer) {
    const int k = (s * kSplit + group) * 128;
    const uint32_t to = lds + (group * kStages + buffer) * kBytes;
    stage_u.copy(from_u, to, k, a.inputs);
    stage_w.copy(from_w, to + kM * 128, k, a.inputs);
  };
  // operand rows of this lane: its output row m of a 32-row product is such that
  // the sixteen results it gets are sixteen outputs side by side
  const int r32 = lane & 31, half = lane >> 5;
  const int wr = 16 * ((r32 >> 2) & 1) + 4 * (r32 >> 3) + (r32 & 3);
  const int wave_m = (wave % kWm) * (kM / kWm), wave_n = (wave / kWm) * (kN / kWn);
  const int at_u = (wave_m + r32) * 128 + ((half ^ turn<false>(r32)) << 4);
  const int at_w = kM * 128 + (wave_n + wr) * 128 + ((half ^ turn<true>(wr)) << 4);
  i32x16 sum[kTn][kTm];
#pragma unroll
  for (int i = 0; i < kTn; ++i)
#pragma unroll
    for (int j = 0; j < kTm; ++j) sum[i][j] = (i32x16)(0);
  // What is copied past the inputs' end are zeros, that no step reads: so many copies
  // are under way at every step.
  const int steps = (a.inputs + kSplit * 128 - 1) / (kSplit * 128);
  constexpr int kEarly = kStages - 1;
#pragma unroll
  for (int s = 0; s < kEarly; ++s) copy(s, s);
  for (int s = 0, at = 0, to = kEarly; s < steps; ++s) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kEarly - 1) * kCopies) : "memory");
    __syncthreads();
    const char* mem = s_mem + (group * kStages + at) * kBytes;
    at = at + 1 == kStages ? 0 : at + 1;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      i32x4 w[kTn], u[kTm];
#pragma unroll
      for (int i = 0; i < kTn; ++i)
        w[i] = *(const i32x4*)(mem + (at_w ^ (ks * 32)) + i * 32 * 128);
#pragma unroll
      for (int j = 0; j < kTm; ++j)
        u[j] = *(const i32x4*)(mem + (at_u ^ (ks * 32)) + j * 32 * 128);
      // the first reads are on their way before the copies are
      if (ks == 0) copy(s + kEarly, to);
#pragma unroll
      for (int i = 0; i < kTn; ++i)
#pragma unroll
        for (int j = 0; j < kTm; ++j)
          sum[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], u[j], sum[i][j], 0, 0, 0);
    }
    to = to + 1 == kStages ? 0 : to + 1;
  }
  // Results go through LDS, 32 rows by 128 bytes of a wavefront at a time, so that
  // whole lines are written.  A row there is 16 bytes longer: sixteen rows fall on
  // different banks.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  constexpr int kAcross = kTn * 32 * (int)sizeof(T) < 128 ? kTn : 4 / (int)sizeof(T);
  constexpr int kRowBytes = kAcross * 32 * (int)sizeof(T), kLong = kRowBytes + 16;
  constexpr int kChunks = kRowBytes / 16, kTall = 64 / kChunks, kEach = 16 / (int)sizeof(T);
  char* const mem = s_mem + wave * 32 * kLong;
  constexpr int kParts = kTn * kTm * 4;
  const auto part_of = [&](int p) {
    const i32x16& x = sum[p / 4 / kTm][p / 4 % kTm];
    const int i = p % 4 * 4;
    return i32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
  };
  if constexpr (kSplit > 1) {
    // the groups' sums meet behind the place of the results
    i32x4* const all = (i32x4*)(s_mem + kWaves * 32 * kLong) + wave * kParts * 64 + lane;
    if (group > 0) {
#pragma unroll
      for (int p = 0; p < kParts; ++p)
        all[((group - 1) * kWaves * kParts + p) * 64] = part_of(p);
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < kSplit - 1; ++g)
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const i32x4 x = all[(g * kWaves * kParts + p) * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[p / 4 / kTm][p / 4 % kTm][p % 4 * 4 + i] += x[i];
      }
  }
  // scales and biases of all this lane's results, in one round trip
  float scale[kTm], w_scale[kTn][16], bias[kTn][16];
#pragma unroll
  for (int j = 0; j < kTm; ++j) {
    const int64_t m = m0 + wave_m + 32 * j + r32;
    scale[j] = a.u_scale[m < a.rows ? m : a.rows - 1];
  }
#pragma unroll
  for (int i = 0; i < kTn; ++i)
#pragma unroll
    for (int e = 0; e < 16; e += 8) {
      // outputs are a multiple of 8
      const int n = min(n0 + wave_n + 32 * i + 16 * half + e, a.outputs - 8);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        w_scale[i][e + x] = a.w_scale[n + x];
        bias[i][e + x] = a.bias ? a.bias[n + x] : 0.0f;
      }
    }
  static_assert(kWaves * (32 * kLong + (kSplit - 1) * kParts * 1024) <= kSplit * kStages * kBytes,
                "the tiles' place holds the results");
#pragma unroll
  for (int j = 0; j < kTm; ++j) {
    const int64_t first = m0 + wave_m + 32 * j;
#pragma unroll
    for (int i0 = 0; i0 < kTn; i0 += kAcross) {
#pragma unroll
      for (int i = i0; i < i0 + kAcross; ++i) {
#pragma unroll
        for (int g = 0; g < 16 / kEach; ++g) {
          float v[kEach];
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            const int x = g * kEach + e;
            v[e] = (float)sum[i][j][x] * (scale[j] * w_scale[i][x]);
            if (a.bias) v[e] += bias[i][x];
          }
          store_elems((T*)(mem + r32 * kLong) + (i - i0) * 32 + 16 * half + g * kEach, v);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int r = 0; r < 32; r += kTall) {
        const int row = r + lane / kChunks, at = lane % kChunks;
        const int n = n0 + wave_n + 32 * i0 + at * kEach;
        const u32x4 x = *(const u32x4*)(mem + row * kLong + at * 16);
        if (first + row < a.rows && n < a.outputs)
          *(u32x4*)((T*)a.y + (first + row) * a.y_row + n) = x;
      }
    }
  }
}

namespace {

template <typename T>
hipError_t quantize(int64_t rows, int64_t channels, const gs_rows& x, int8_t* codes,
                    float* scales, hipStream_t s) {
  // a row by a wavefront keeps its elements in registers up to 2,048 channels
  if (channels <= 2048)
    return launch_all((rows + 3) / 4, 256, [&](uint32_t first, dim3 n) {
      quantize_rows_kernel<T, 64><<<n, 256, 0, s>>>(rows, (int)channels, (const T*)x.data, x.row,
                                                    codes, scales, first);
    });
  return launch_all(rows, 256, [&](uint32_t first, dim3 n) {
    quantize_rows_kernel<T, 256><<<n, 256, 0, s>>>(rows, (int)channels, (const T*)x.data, x.row,
                                                   codes, scales, first);
  });
}

template <typename T, int kWaves, bool kOwn>
hipError_t few(const LinearArgs& a, hipStream_t s) {
  linear_few_kernel<T, kWaves, kOwn>
      <<<dim3((a.outputs + 15) / 16), kWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int kM, int kN, int kWm, int kWn, int kStages, int kSplit = 1>
hipError_t many(LinearArgs a, hipStream_t s) {
  a.tiles_n = (uint32_t)((a.outputs + kN - 1) / kN);
  a.tiles = (uint32_t)((a.rows + kM - 1) / kM) * a.tiles_n;
  linear_many_kernel<T, kM, kN, kWm, kWn, kStages, kSplit>
      <<<dim3((a.tiles + 7) / 8 * 8), kWm * kWn * kSplit * 64, 0, s>>>(a);
  return hipGetLastError();
}

// Whether workgroups bring the rows to codes themselves: where that is little work
// for all of them together (us with a launch for the codes : without; inputs by
// outputs): one row of 4,096 by 4,096 9.8 : 7.3, of 16,384 by 4,096 26.3 : 18.9;
// four of 4,096 by 4,096 10.3 : 9.0; eight of 1,024 by 1,024 6.1 : 4.7.  The limit is
// where the two meet with weights from a cache (eight of 4,096 by 4,096 10.7 : 11.0, of
// 2,048 by 8,192 10.9 : 12.4); from memory 10.8 : 10.7 and 12.2 : 10.1.
bool own_codes(int64_t rows, int64_t inputs, int64_t outputs) {
  const int64_t shares = rows <= 2 ? rows : rows <= 4 ? 4 : 8;
  return rows <= 8 && shares * inputs <= (outputs <= kOutputsOf16 ? kOwnElems<16> : kOwnElems<8>) &&
         shares * inputs * outputs <= (int64_t)96 << 20;
}

template <typename T>
hipError_t linear(const LinearArgs& a, hipStream_t s) {
  const bool of16 = a.outputs <= kOutputsOf16;
  if (own_codes(a.rows, a.inputs, a.outputs))
    return of16 ? few<T, 16, true>(a, s) : few<T, 8, true>(a, s);
  const auto tiles = [&](int64_t tall, int64_t wide) {
    return ((a.rows + tall - 1) / tall) * ((a.outputs + wide - 1) / wide);
  };
  // us, few rows : tiles of 64 x 32 outputs: 16 rows of 8,192 by 2,048 15.7 : 18.3, of
  // 4,096 by 4,096 11.7 : 13.3; with more outputs every workgroup's reading of all
  // rows weighs more (16 of 8,192 by 8,192 26.5 : 21.7).
  if (a.rows <= 16 && of16) return few<T, 16, false>(a, s);
  // Small tiles while all run at a time and wait for memory and for each other's
  // steps: the steps shared by four groups of wavefronts, by two, by none (us of the
  // three: 64 rows of 4,096 by 4,096 15.1, 17.2, 19.4; 200 of them 20.5, 15.9, 19.3;
  // 1,024 of 2,048 by 2,048 28.6, 20.6, 17.7).
  if (tiles(64, 32) <= kUnits) return many<T, 64, 32, 2, 1, 3, 4>(a, s);
  if (tiles(64, 64) <= kUnits) return many<T, 64, 64, 2, 2, 3, 2>(a, s);
  if (tiles(64, 64) <= 2 * kUnits) return many<T, 64, 64, 2, 2, 3>(a, s);
  // A tile a compute unit: two steps on their way, or two workgroups with one each
  // (2,048 rows of 2,048 by 2,048 21.7 : 25.3; with more tiles, 4,096 such rows,
  // 37.1 : 33.5).
  const int64_t n128 = tiles(128, 128);
  if (n128 <= kUnits) return many<T, 128, 128, 2, 2, 3>(a, s);
  // Else the form whose last tiles end first: a unit takes about 10, 25 and 32 us
  // for a tile of 128 x 128, 192 x 256 and 256 x 256 with 2,048 inputs (us of the
  // three, rows by outputs: 1,024 by 8,192 30.5, 34.4, 39.4; 1,500 by 8,192 47.3, 37.3,
  // 40.1; 4,096 by 4,096 55.4, 57.5, 46.5; 9,000 by 4,096 108, 101, 107).
  const auto turns = [](int64_t n) { return (n + kUnits - 1) / kUnits; };
  const int64_t t128 = 10 * turns(n128), t192 = 25 * turns(tiles(192, 256)),
                t256 = 32 * turns(tiles(256, 256));
  if (t256 < t128 && t256 <= t192) return many<T, 256, 256, 2, 4, 2>(a, s);
  if (t192 < t128) return many<T, 192, 256, 2, 4, 2>(a, s);
  return many<T, 128, 128, 2, 2, 2>(a, s);
}

size_t codes_bytes(int64_t rows, int64_t channels) {
  return ((size_t)rows * channels + 255) / 256 * 256;
}

}  // namespace
}  // namespace gs

extern "C" {

size_t gs_linear_i8_bytes(const gs_linear_config& cfg, int64_t rows) {
  return gs::own_codes(rows, cfg.inputs, cfg.outputs) ? 0
                                         : gs::codes_bytes(rows, cfg.inputs) + (size_t)rows * 4;
}

hipError_t gs_launch_quantize_rows(int32_t dtype, int64_t rows, int64_t channels,
                                   const gs_rows& x, int8_t* codes, float* scales,
                                   hipStream_t s) {
  if (dtype == GS_F32) return gs::quantize<float>(rows, channels, x, codes, scales, s);
  if (dtype == GS_BF16) return gs::quantize<gs::Bf16>(rows, channels, x, codes, scales, s);
  return gs::quantize<gs::F16>(rows, channels, x, codes, scales, s);
}

hipError_t gs_launch_linear_i8(const gs_linear_config& cfg, int64_t rows, const gs_rows& x,
                               const int8_t* w, const float* w_scale, const float* bias,
                               const gs_rows& y, void* workspace, hipStream_t s) {
  int8_t* u = (int8_t*)workspace;
  float* u_scale = (float*)(u + gs::codes_bytes(rows, cfg.inputs));
  if (!gs::own_codes(rows, cfg.inputs, cfg.outputs)) {
    const hipError_t e = gs_launch_quantize_rows(cfg.dtype, rows, cfg.inputs, x, u, u_scale, s);
    if (e != hipSuccess) return e;
  }
  gs::LinearArgs a = {};
  a.rows = rows;
  a.inputs = (int)cfg.inputs;
  a.outputs = (int)cfg.outputs;
  a.x = x.data;
  a.x_row = x.row;
  a.u = u;
  a.u_scale = u_scale;
  a.w = w;
  a.w_scale = w_scale;
  a.bias = bias;
  a.y = y.data;
  a.y_row = y.row;
  if (cfg.dtype == GS_F32) return gs::linear<float>(a, s);
  if (cfg.dtype == GS_BF16) return gs::linear<gs::Bf16>(a, s);
  return gs::linear<gs::F16>(a, s);
}

}  // extern "C"
