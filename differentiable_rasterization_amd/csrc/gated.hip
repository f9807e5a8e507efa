// gated.hip — gated linear recurrence over documents, and its gradient.
//
//   a = sigmoid(gate),  h_t = a_t h_{t-1} + u_t,
//   u_t = (1 - a_t) x_t (coupled: the over operator with alpha = 1 - a) or x_t.
//
// Backward, from the last step: g_t = dy_t + a_{t+1} g_{t+1};
//   dx = (1 - a) g or g,  dgate = g (h_{t-1} - x_t) a (1 - a) or
//   g h_{t-1} a (1 - a);  the first step sends a g to the state it took in.
//
// A step costs a dozen operations on six to twelve bytes, so memory traffic
// should bound the operator; what stands in the way is that the steps depend on
// each other.  The recurrence is a composition of maps h -> A h + H, which is
// associative, so each document is cut into chunks whose maps are formed at
// the same time.
//   Documents of at most 64 steps: a wavefront walks a document.
//   Otherwise, one pass over the data: a workgroup keeps its chunk's inputs in
//   registers, composes its map, publishes it, composes the maps of the chunks
//   before it in its document as they appear, and runs its steps from the
//   state that gives.  Every workgroup reads all earlier maps (eight bytes
//   a channel each), so nobody waits for more than a map, and the maps are
//   composed in one order whatever the timing.
//   Documents of more chunks than that is worth: three passes (chunk maps;
//   per channel, the state every chunk starts from; the steps).
// The order of every sum is fixed, so results are the same bits every time.
// Lanes run over channels, wavefronts over steps; states are fp32 throughout,
// and only the outputs are rounded, once.
//
// The backward needs h_{t-1} in fp32: reading it from the rounded outputs
// would put their rounding into the gate's gradient.  The forward therefore
// keeps the state before every 16th step, and the backward runs 16 steps
// forward from it in registers before it runs them back.
#include "tokens.h"

namespace gs {

constexpr int kChunk = 64;  // steps of a chunk
constexpr int kSub = 16;    // steps between saved states

struct GatedArgs {
  Docs docs;
  int channels, groups;  // groups: wavefronts over the channels
  int coupled;
  const void* gate;
  const void* x;
  const void* dy;
  int64_t gate_row, x_row, dy_row;
  void* y;      // forward
  void* dgate;  // backward
  void* dx;
  int64_t y_row, dgate_row, dx_row;
  const float* state_in;  // forward: state; backward: its gradient from the end
  float* state_out;       // forward: state; backward: gradient to the start
  float* saved;
  float* maps;   // [chunk][channels] A
  float* carry;  // [chunk][channels] H, then the state the chunk starts from
  uint32_t chunks;  // bound on the number of chunks
  uint32_t block0;  // chunks' states: first workgroup of the launch
};

// a = sigmoid(f) and z = 1 - a, both accurate relative to themselves (a gate
// that is nearly open has a tiny z, a shut one a tiny a).  fp32 inputs carry
// the exponent's rounding along; of 16-bit ones it is 2^-24 |f| beside the 2^-9 or
// 2^-12 |f| that f itself was rounded by, and is left.
template <bool kExact>
__device__ inline void gate_of(float f, float& a, float& z) {
  float m;
  if constexpr (kExact) {
    const float v = fabsf(f) > 128.0f ? 128.0f : fabsf(f);  // keeps NaN
    const float t = -v * kLog2e;
    m = __builtin_amdgcn_exp2f(t);
    m = fmaf(m, fmaf(-v, kLog2e, -t) * kLn2, m);
  } else {
    m = __builtin_amdgcn_exp2f(fabsf(f) * -kLog2e);
  }
  const float r = __builtin_amdgcn_rcpf(1.0f + m);
  const float small = m * r, big = 1.0f - small;
  a = f >= 0.0f ? big : small;
  z = f >= 0.0f ? small : big;
}

template <typename T>
__device__ inline const T* row_ptr(const void* p, int64_t row, int64_t stride, int ch) {
  return (const T*)p + row * stride + ch;
}

// Work item of this wavefront: (chunk or document, channel group).
struct Item {
  int doc;          // -1: none
  uint32_t chunk;   // index over all documents' chunks
  int64_t row0;     // first row
  int steps;
  int ch;           // the lane's first channel
  bool on;          // the lane has channels
};

template <int V>
__device__ inline Item chunk_item(const GatedArgs& a) {
  Item it;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t unit = __builtin_amdgcn_readfirstlane((uint32_t)(w / a.groups));
  const int group = __builtin_amdgcn_readfirstlane((int)(w % a.groups));
  uint32_t local, n;
  it.doc = -1;
  if (unit >= a.chunks) return it;
  Doc d;
  it.doc = find_document<false>(a.docs, 1, kChunk, unit, &local, &n, &d, false);
  if (it.doc < 0) return it;
  it.chunk = unit;
  it.row0 = (int64_t)d.qs + (int64_t)local * kChunk;
  it.steps = min(kChunk, d.ql - (int)local * kChunk);
  it.ch = (group * 64 + (threadIdx.x & 63)) * V;
  it.on = it.ch < a.channels;
  return it;
}

// 1. The chunk's map: A = product of a, H = the state it makes from zero.
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_maps_kernel(GatedArgs a) {
  const Item it = chunk_item<V>(a);
  if (it.doc < 0 || !it.on) return;
  constexpr bool kExact = __is_same(T, float);
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
  }
  const T* pf = row_ptr<T>(a.gate, it.row0, a.gate_row, it.ch);
  const T* px = row_ptr<T>(a.x, it.row0, a.x_row, it.ch);
#pragma unroll 8
  for (int t = 0; t < it.steps; ++t) {
    float f[V], x[V];
    load_elems(pf + t * a.gate_row, f);
    load_elems(px + t * a.x_row, x);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g, z;
      gate_of<kExact>(f[v], g, z);
      A[v] *= g;
      H[v] = fmaf(g, H[v], a.coupled ? z * x[v] : x[v]);
    }
  }
  store_elems(a.maps + (int64_t)it.chunk * a.channels + it.ch, A);
  store_elems(a.carry + (int64_t)it.chunk * a.channels + it.ch, H);
}

// 1, backward: the map of the message e_t = a_t (dy_t + e_{t+1}).
template <typename T, int V>
__global__ __launch_bounds__(256) void gated_maps_bwd_kernel(GatedArgs a) {
  const Item it = chunk_item<V>(a);
  if (it.doc < 0 || !it.on) return;
  constexpr bool kExact = __is_same(T, float);
  float A[V], E[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    E[v] = 0.0f;
  }
  const T* pf = row_ptr<T>(a.gate, it.row0, a.gate_row, it.ch);
  const T* pd = row_ptr<T>(a.dy, it.row0, a.dy_row, it.ch);
#pragma unroll 8
  for (int t = it.steps - 1; t >= 0; --t) {
    float f[V], d[V];
    load_elems(pf + t * a.gate_row, f);
    load_elems(pd + t * a.dy_row, d);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float g, z;
      gate_of<kExact>(f[v], g, z);
      A[v] *= g;
      E[v] = g * (d[v] + E[v]);
    }
  }
  store_elems(a.maps + (int64_t)it.chunk * a.channels + it.ch, A);
  store_elems(a.carry + (int64_t)it.chunk * a.channels + it.ch, E);
}

// 2. The state every chunk of a document starts from (backward: the message
// it receives, chunks from the last).  16 channels a workgroup, S lanes a
// channel: each composes its share of the chunks, the shares are applied in
// order, and each lane walks its share again.
template <bool kBack, int S>
__global__ __launch_bounds__(16 * S) void gated_carry_kernel(GatedArgs a) {
  __shared__ float s_a[S][17], s_h[S][17];
  const int per = (a.channels + 15) / 16;
  const uint32_t block = a.block0 + blockIdx.x;
  const int doc = block / per;
  const int c = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int ch = (block % per) * 16 + c;
  const uint32_t base = units_before(a.docs.q_start, a.docs.q_len, a.docs.rows_q, doc, kChunk);
  const int len = clamp_len(a.docs.q_start[doc], a.docs.q_len[doc], a.docs.rows_q);
  const int n = (len + kChunk - 1) / kChunk;
  if (base + n > a.chunks) return;  // documents that share rows: no room for their maps
  const bool on = ch < a.channels;
  const int lo = (int)((int64_t)n * seg / S), hi = (int)((int64_t)n * (seg + 1) / S);
  float h = on && a.state_in ? a.state_in[(int64_t)doc * a.channels + ch] : 0.0f;
  float A = 1.0f, H = 0.0f;
  if (on) {
#pragma unroll 4
    for (int i = lo; i < hi; ++i) {
      const int64_t o = (int64_t)(base + (kBack ? n - 1 - i : i)) * a.channels + ch;
      const float m = a.maps[o];
      H = fmaf(m, H, a.carry[o]);
      A *= m;
    }
  }
  s_a[seg][c] = A;
  s_h[seg][c] = H;
  __syncthreads();
  if (!on) return;
#pragma unroll 8
  for (int i = 0; i < seg; ++i) h = fmaf(s_a[i][c], h, s_h[i][c]);
#pragma unroll 4
  for (int i = lo; i < hi; ++i) {
    const int64_t o = (int64_t)(base + (kBack ? n - 1 - i : i)) * a.channels + ch;
    const float m = a.maps[o], H = a.carry[o];
    a.carry[o] = h;
    h = fmaf(m, h, H);
  }
  if (seg == S - 1 && a.state_out) a.state_out[(int64_t)doc * a.channels + ch] = h;
}

// The whole document of this wavefront, for the one-launch form.
template <int V>
__device__ inline Item doc_item(const GatedArgs& a, bool want_chunk) {
  Item it;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int doc = __builtin_amdgcn_readfirstlane((int)(w / a.groups));
  const int group = __builtin_amdgcn_readfirstlane((int)(w % a.groups));
  it.doc = doc < a.docs.count ? doc : -1;
  if (it.doc < 0) return it;
  const int start = a.docs.q_start[doc];
  it.steps = clamp_len(start, a.docs.q_len[doc], a.docs.rows_q);
  it.row0 = clamp_start(start, a.docs.rows_q);
  it.chunk = want_chunk ? units_before(a.docs.q_start, a.docs.q_len, a.docs.rows_q, doc, kChunk)
                        : 0;
  if (want_chunk && it.chunk + (it.steps + kChunk - 1) / kChunk > a.chunks) it.doc = -1;
  it.ch = (group * 64 + (threadIdx.x & 63)) * V;
  it.on = it.ch < a.channels;
  return it;
}

// 3. The steps of a chunk (kDirect: of a document) from the state it starts
// from.
template <typename T, int V, bool kDirect>
__global__ __launch_bounds__(256) void gated_run_kernel(GatedArgs a) {
  const Item it = kDirect ? doc_item<V>(a, a.saved != nullptr) : chunk_item<V>(a);
  if (it.doc < 0 || !it.on) return;
  constexpr bool kExact = __is_same(T, float);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  const int64_t so = (int64_t)it.doc * a.channels + it.ch;
  if constexpr (kDirect) {
    if (a.state_in) load_elems(a.state_in + so, h);
  } else {
    load_elems(a.carry + (int64_t)it.chunk * a.channels + it.ch, h);
  }
  const T* pf = row_ptr<T>(a.gate, it.row0, a.gate_row, it.ch);
  const T* px = row_ptr<T>(a.x, it.row0, a.x_row, it.ch);
  T* py = (T*)a.y + it.row0 * a.y_row + it.ch;
  float* save = a.saved ? a.saved + (int64_t)it.chunk * (kChunk / kSub) * a.channels + it.ch
                        : nullptr;
  for (int t0 = 0; t0 < it.steps; t0 += kSub) {
    if (save) store_elems(save + (int64_t)(t0 / kSub) * a.channels, h);
    const int end = min(it.steps, t0 + kSub);
#pragma unroll 8
    for (int t = t0; t < end; ++t) {
      float f[V], x[V];
      load_elems(pf + t * a.gate_row, f);
      load_elems(px + t * a.x_row, x);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float g, z;
        gate_of<kExact>(f[v], g, z);
        h[v] = fmaf(g, h[v], a.coupled ? z * x[v] : x[v]);
      }
      store_elems(py + t * a.y_row, h);
    }
  }
  if constexpr (kDirect) {
    if (a.state_out) store_elems(a.state_out + so, h);
  }
}

// 3, backward: 16 steps at a time from the last, forward from the saved state
// in registers, then back.
template <typename T, int V, bool kDirect>
__global__ __launch_bounds__(256) void gated_run_bwd_kernel(GatedArgs a) {
  const Item it = kDirect ? doc_item<V>(a, true) : chunk_item<V>(a);
  if (it.doc < 0 || !it.on) return;
  constexpr bool kExact = __is_same(T, float);
  float e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = 0.0f;
  const int64_t so = (int64_t)it.doc * a.channels + it.ch;
  if constexpr (kDirect) {
    if (a.state_in) load_elems(a.state_in + so, e);
  } else {
    load_elems(a.carry + (int64_t)it.chunk * a.channels + it.ch, e);
  }
  const float* save = a.saved + (int64_t)it.chunk * (kChunk / kSub) * a.channels + it.ch;
  for (int sub = (it.steps - 1) / kSub; sub >= 0 && it.steps > 0; --sub) {
    const int64_t row = it.row0 + sub * kSub;
    const int n = min(kSub, it.steps - sub * kSub);
    const T* pf = row_ptr<T>(a.gate, row, a.gate_row, it.ch);
    const T* px = row_ptr<T>(a.x, row, a.x_row, it.ch);
    const T* pd = row_ptr<T>(a.dy, row, a.dy_row, it.ch);
    T* of = (T*)a.dgate + row * a.dgate_row + it.ch;
    T* ox = (T*)a.dx + row * a.dx_row + it.ch;
    float before[kSub][V], f[kSub][V], x[kSub][V], d[kSub][V];
    float h[V];
    load_elems(save + (int64_t)sub * a.channels, h);
#pragma unroll
    for (int t = 0; t < kSub; ++t) {
      if (t < n) {
        load_elems(pf + t * a.gate_row, f[t]);
        load_elems(px + t * a.x_row, x[t]);
        load_elems(pd + t * a.dy_row, d[t]);
      }
    }
#pragma unroll
    for (int t = 0; t < kSub; ++t) {
      if (t < n) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g, z;
          gate_of<kExact>(f[t][v], g, z);
          before[t][v] = h[v];
          h[v] = fmaf(g, h[v], a.coupled ? z * x[t][v] : x[t][v]);
        }
      }
    }
#pragma unroll
    for (int t = kSub - 1; t >= 0; --t) {
      if (t < n) {
        float df[V], dx[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g, z;
          gate_of<kExact>(f[t][v], g, z);
          const float up = d[t][v] + e[v];
          dx[v] = a.coupled ? up * z : up;
          df[v] = up * (a.coupled ? before[t][v] - x[t][v] : before[t][v]) * (g * z);
          e[v] = g * up;
        }
        store_elems(of + t * a.dgate_row, df);
        store_elems(ox + t * a.dx_row, dx);
      }
    }
  }
  if constexpr (kDirect) {
    if (a.state_out) store_elems(a.state_out + so, e);
  }
}

// ---------------------------------------------------------------------------
// One pass
// ---------------------------------------------------------------------------
constexpr int kPassWaves = 8;
// A published map is one 64-bit word a channel, (A, H), so that it needs no
// flag beside it; all bits set is "not yet" (a NaN is stored as another NaN).
constexpr uint64_t kNoMap = ~(uint64_t)0;

__device__ inline uint64_t map_word(float a, float h) {
  if (a != a) a = __builtin_nanf("");
  if (h != h) h = __builtin_nanf("");
  return (uint64_t)__builtin_bit_cast(uint32_t, a) << 32 | __builtin_bit_cast(uint32_t, h);
}

// Clears the maps and the ticket, and takes a copy of the states, since the
// last chunk of a document may replace them (state_out may be state_in) before
// the first has read them; hands an empty document's state through.
__global__ __launch_bounds__(256) void gated_clear_kernel(GatedArgs a, uint64_t* maps,
                                                          int64_t words, uint32_t* ticket,
                                                          float* states_in) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t k = i; k < words; k += step) maps[k] = kNoMap;
  if (i == 0) *ticket = 0;
  const int64_t states = (int64_t)a.docs.count * a.channels;
  for (int64_t k = i; k < states; k += step) {
    const float h = a.state_in ? a.state_in[k] : 0.0f;
    states_in[k] = h;
    const int doc = (int)(k / a.channels);
    if (a.state_out && clamp_len(a.docs.q_start[doc], a.docs.q_len[doc], a.docs.rows_q) == 0)
      a.state_out[k] = h;
  }
}

// A 32-bit word of a row: two 16-bit channels or one fp32.
template <typename T>
struct Pack {
  static constexpr int V = 4 / sizeof(T);
};
template <typename T>
__device__ inline void open_word(uint32_t w, float (&v)[Pack<T>::V]) {
  if constexpr (__is_same(T, float)) v[0] = __builtin_bit_cast(float, w);
  else unpack2<T>(w, v[0], v[1]);
}
template <typename T>
__device__ inline uint32_t close_word(const float (&v)[Pack<T>::V]) {
  if constexpr (__is_same(T, float)) return __builtin_bit_cast(uint32_t, v[0]);
  else return pack2<T>(v[0], v[1]);
}

// The workgroup's chunk, by ticket: tickets are taken in the order workgroups
// start, so every chunk that this one waits for has a workgroup that runs and
// itself waits only for earlier ones.
struct PassItem {
  int doc;
  uint32_t unit, local, units;
  uint32_t chunk64;  // index of the document's first chunk of kChunk steps
  Doc d;
  int ch;
  bool on;
};
template <int V, bool kBack>
__device__ inline PassItem pass_item(const GatedArgs& a, uint32_t chunks, int chunk,
                                     uint32_t* ticket) {
  __shared__ uint32_t s_ticket;
  if (threadIdx.x == 0) s_ticket = atomicAdd(ticket, 1u);
  __syncthreads();
  const uint32_t t = __builtin_amdgcn_readfirstlane(s_ticket);
  PassItem it;
  it.doc = -1;
  const uint32_t u = t / (uint32_t)a.groups;
  if (u >= chunks) return it;
  it.unit = kBack ? chunks - 1 - u : u;
  it.ch = ((int)(t % (uint32_t)a.groups) * 64 + (threadIdx.x & 63)) * V;
  it.on = it.ch < a.channels;
  it.doc = find_document<false>(a.docs, 1, (uint32_t)chunk, it.unit, &it.local, &it.units, &it.d,
                                false);
  // documents that share rows have more chunks than there is room for
  if (it.doc >= 0 && it.unit - it.local + it.units > chunks) it.doc = -1;
  it.chunk64 = it.doc < 0 || !a.saved ? 0
                                      : units_before(a.docs.q_start, a.docs.q_len, a.docs.rows_q,
                                                     it.doc, kChunk);
  if (a.saved && it.chunk64 + (it.d.ql + kChunk - 1) / kChunk > a.chunks) it.doc = -1;
  return it;
}

// Composes maps [from, from + step, ...) (n of them) of the lane's channels,
// in that order, after the map (A, H) so far.  Waits are for workgroups that
// are already running (microseconds); the bound, some seconds in all, only ends
// a wait that cannot end, with results that are not numbers.
template <int V>
__device__ inline void compose_maps(const uint64_t* maps, int64_t from, int64_t step, int n,
                                    float (&A)[V], float (&H)[V]) {
  constexpr int kBatch = 8;
  int spins = 1 << 20;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    uint64_t w[kBatch][V];
    while (true) {
      bool all = true;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          w[i][v] = __hip_atomic_load(maps + from + (int64_t)min(i0 + i, n - 1) * step + v,
                                      __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          all = all && w[i][v] != kNoMap;
        }
      }
      if (__ballot(!all) == 0 || --spins <= 0) break;
      __builtin_amdgcn_s_sleep(2);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i < n) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float m = __builtin_bit_cast(float, (uint32_t)(w[i][v] >> 32));
          H[v] = fmaf(m, H[v], __builtin_bit_cast(float, (uint32_t)w[i][v]));
          A[v] *= m;
        }
      }
    }
  }
}

// Forward: STEPS steps of a wavefront's channels in registers, two words each.
// With 32 steps two workgroups fit a compute unit, one loading beside the other's
// steps: 65,536 x 2,048 bf16, 805 MB in 226 us (3.6 TB/s), the call 234; with 64
// steps and one workgroup 262.  Vector instructions issue in 63% of its cycles
// (81 million, each gate is formed twice): 150 us of issue and 158 of bytes, which
// overlap only in part.  fp32 has two thirds as many instructions a byte.
template <typename T, int STEPS>
__global__ __launch_bounds__(64 * kPassWaves, 4) void gated_pass_kernel(GatedArgs a,
                                                                        uint64_t* maps,
                                                                        uint32_t chunks,
                                                                        uint32_t* ticket) {
  constexpr int V = Pack<T>::V, kLong = STEPS * kPassWaves;
  constexpr bool kExact = __is_same(T, float);
  __shared__ float s_a[kPassWaves][64 * V], s_h[kPassWaves][64 * V];
  __shared__ float p_a[kPassWaves][64 * V], p_h[kPassWaves][64 * V];
  const PassItem it = pass_item<V, false>(a, chunks, kLong, ticket);
  if (it.doc < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = (int)it.local * kLong + wave * STEPS;
  const int n = min(STEPS, it.d.ql - t0);
  const int64_t row = (int64_t)it.d.qs + t0;
  uint32_t f[STEPS], x[STEPS];
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
  }
  if (n > 0 && it.on) {
    const T* pf = row_ptr<T>(a.gate, row, a.gate_row, it.ch);
    const T* px = row_ptr<T>(a.x, row, a.x_row, it.ch);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      f[i] = *(const uint32_t*)(pf + min(i, n - 1) * a.gate_row);
      x[i] = *(const uint32_t*)(px + min(i, n - 1) * a.x_row);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      if (i < n) {
        float fv[V], xv[V];
        open_word<T>(f[i], fv);
        open_word<T>(x[i], xv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g, z;
          gate_of<kExact>(fv[v], g, z);
          A[v] *= g;
          H[v] = fmaf(g, H[v], a.coupled ? z * xv[v] : xv[v]);
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s_a[wave][lane * V + v] = A[v];
    s_h[wave][lane * V + v] = H[v];
  }
  __syncthreads();
  const int64_t first = ((int64_t)it.unit - it.local) * a.channels + it.ch;
  if (wave == 0 && it.on && it.local + 1 < it.units) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float ma = 1.0f, mh = 0.0f;
      for (int w = 0; w < kPassWaves; ++w) {
        mh = fmaf(s_a[w][lane * V + v], mh, s_h[w][lane * V + v]);
        ma *= s_a[w][lane * V + v];
      }
      __hip_atomic_store(maps + first + (int64_t)it.local * a.channels + v, map_word(ma, mh),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  // the chunks before this one, shared out among the wavefronts in order
  const int lo = (int)it.local * wave / kPassWaves, hi = (int)it.local * (wave + 1) / kPassWaves;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    H[v] = 0.0f;
  }
  if (it.on && hi > lo)
    compose_maps<V>(maps, first + (int64_t)lo * a.channels, a.channels, hi - lo, A, H);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p_a[wave][lane * V + v] = A[v];
    p_h[wave][lane * V + v] = H[v];
  }
  __syncthreads();
  if (n <= 0 || !it.on) return;
  float h[V];
  const int64_t so = (int64_t)it.doc * a.channels + it.ch;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = a.state_in ? a.state_in[so + v] : 0.0f;
    for (int w = 0; w < kPassWaves; ++w)
      h[v] = fmaf(p_a[w][lane * V + v], h[v], p_h[w][lane * V + v]);
    for (int w = 0; w < wave; ++w)
      h[v] = fmaf(s_a[w][lane * V + v], h[v], s_h[w][lane * V + v]);
  }
  T* py = (T*)a.y + row * a.y_row + it.ch;
  float* save = nullptr;
  if (a.saved) {
    const int64_t chunk = (int64_t)it.chunk64 + t0 / kChunk;
    save = a.saved + (chunk * (kChunk / kSub) + t0 % kChunk / kSub) * a.channels + it.ch;
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (i < n) {
      if (i % kSub == 0 && save) {
#pragma unroll
        for (int v = 0; v < V; ++v) save[(int64_t)(i / kSub) * a.channels + v] = h[v];
      }
      float fv[V], xv[V];
      open_word<T>(f[i], fv);
      open_word<T>(x[i], xv);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float g, z;
        gate_of<kExact>(fv[v], g, z);
        h[v] = fmaf(g, h[v], a.coupled ? z * xv[v] : xv[v]);
      }
      *(uint32_t*)(py + i * a.y_row) = close_word<T>(h);
    }
  }
  if (a.state_out && t0 + n == it.d.ql) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.state_out[so + v] = h[v];
  }
}

// Backward: the same from the other end, three words a step.  20,011 x 1,024
// fp32 of 12 documents: 100 us after a forward of 61 (410 and 246 MB and the saved
// states: 4.3 TB/s with what the forward left in cache).
template <typename T, int STEPS>
__global__ __launch_bounds__(64 * kPassWaves, 2) void gated_pass_bwd_kernel(GatedArgs a,
                                                                            uint64_t* maps,
                                                                            uint32_t chunks,
                                                                            uint32_t* ticket) {
  constexpr int V = Pack<T>::V, kLong = STEPS * kPassWaves;
  constexpr bool kExact = __is_same(T, float);
  __shared__ float s_a[kPassWaves][64 * V], s_h[kPassWaves][64 * V];
  __shared__ float p_a[kPassWaves][64 * V], p_h[kPassWaves][64 * V];
  const PassItem it = pass_item<V, true>(a, chunks, kLong, ticket);
  if (it.doc < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = (int)it.local * kLong + wave * STEPS;
  const int n = min(STEPS, it.d.ql - t0);
  const int64_t row = (int64_t)it.d.qs + t0;
  uint32_t f[STEPS], x[STEPS], d[STEPS];
  float A[V], E[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    E[v] = 0.0f;
  }
  if (n > 0 && it.on) {
    const T* pf = row_ptr<T>(a.gate, row, a.gate_row, it.ch);
    const T* px = row_ptr<T>(a.x, row, a.x_row, it.ch);
    const T* pd = row_ptr<T>(a.dy, row, a.dy_row, it.ch);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      f[i] = *(const uint32_t*)(pf + min(i, n - 1) * a.gate_row);
      d[i] = *(const uint32_t*)(pd + min(i, n - 1) * a.dy_row);
      x[i] = *(const uint32_t*)(px + min(i, n - 1) * a.x_row);
    }
#pragma unroll
    for (int i = STEPS - 1; i >= 0; --i) {
      if (i < n) {
        float fv[V], dv[V];
        open_word<T>(f[i], fv);
        open_word<T>(d[i], dv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g, z;
          gate_of<kExact>(fv[v], g, z);
          A[v] *= g;
          E[v] = g * (dv[v] + E[v]);
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s_a[wave][lane * V + v] = A[v];
    s_h[wave][lane * V + v] = E[v];
  }
  __syncthreads();
  const int64_t first = ((int64_t)it.unit - it.local) * a.channels + it.ch;
  if (wave == 0 && it.on && it.local > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float ma = 1.0f, mh = 0.0f;
      for (int w = kPassWaves - 1; w >= 0; --w) {
        mh = fmaf(s_a[w][lane * V + v], mh, s_h[w][lane * V + v]);
        ma *= s_a[w][lane * V + v];
      }
      __hip_atomic_store(maps + first + (int64_t)it.local * a.channels + v, map_word(ma, mh),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  // the chunks after this one, from the last, shared out among the wavefronts
  const int after = (int)(it.units - 1 - it.local);
  const int lo = after * wave / kPassWaves, hi = after * (wave + 1) / kPassWaves;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.0f;
    E[v] = 0.0f;
  }
  if (it.on && hi > lo)
    compose_maps<V>(maps, first + (int64_t)((int)it.units - 1 - lo) * a.channels, -a.channels,
                    hi - lo, A, E);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p_a[wave][lane * V + v] = A[v];
    p_h[wave][lane * V + v] = E[v];
  }
  __syncthreads();
  if (n <= 0 || !it.on) return;
  float e[V];
  const int64_t so = (int64_t)it.doc * a.channels + it.ch;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = a.state_in ? a.state_in[so + v] : 0.0f;
    for (int w = 0; w < kPassWaves; ++w)
      e[v] = fmaf(p_a[w][lane * V + v], e[v], p_h[w][lane * V + v]);
    for (int w = kPassWaves - 1; w > wave; --w)
      e[v] = fmaf(s_a[w][lane * V + v], e[v], s_h[w][lane * V + v]);
  }
  T* of = (T*)a.dgate + row * a.dgate_row + it.ch;
  T* ox = (T*)a.dx + row * a.dx_row + it.ch;
  const int64_t chunk = (int64_t)it.chunk64 + t0 / kChunk;
  const float* save =
      a.saved + (chunk * (kChunk / kSub) + t0 % kChunk / kSub) * a.channels + it.ch;
#pragma unroll
  for (int sub = STEPS / kSub - 1; sub >= 0; --sub) {
    if (sub * kSub < n) {
      float before[kSub][V], h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = save[(int64_t)sub * a.channels + v];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const int i = sub * kSub + j;
        float fv[V], xv[V];
        open_word<T>(f[i], fv);
        open_word<T>(x[i], xv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float g, z;
          gate_of<kExact>(fv[v], g, z);
          before[j][v] = h[v];
          h[v] = fmaf(g, h[v], a.coupled ? z * xv[v] : xv[v]);
        }
      }
#pragma unroll
      for (int j = kSub - 1; j >= 0; --j) {
        const int i = sub * kSub + j;
        if (i < n) {
          float fv[V], xv[V], dv[V], df[V], dx[V];
          open_word<T>(f[i], fv);
          open_word<T>(x[i], xv);
          open_word<T>(d[i], dv);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float g, z;
            gate_of<kExact>(fv[v], g, z);
            const float up = dv[v] + e[v];
            dx[v] = a.coupled ? up * z : up;
            df[v] = up * (a.coupled ? before[j][v] - xv[v] : before[j][v]) * (g * z);
            e[v] = g * up;
          }
          *(uint32_t*)(of + i * a.dgate_row) = close_word<T>(df);
          *(uint32_t*)(ox + i * a.dx_row) = close_word<T>(dx);
        }
      }
    }
  }
  if (a.state_out && t0 == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.state_out[so + v] = e[v];
  }
}

}  // namespace gs

using namespace gs;

namespace {

uint32_t chunk_bound(int64_t rows, int32_t count) {
  return (uint32_t)(rows / kChunk + count);
}

// Which form a call takes.  kPass: up to 1024 chunks, since every workgroup
// reads the maps before it.  One pass against three, forward and backward of a
// document: 131,072 x 1,024 bf16 291 and 492 us against 307 and 782, fp32 402
// and 657 against 557 and 768; 262,144 x 512 bf16 367 and 560 against 319 and
// 786, fp32 437 and 730 against 588 and 785.  Past that the maps, which grow
// with the square, cost more than a pass over the inputs.
enum Form { kDirectForm, kPassForm, kThreeForm };
constexpr int kPassFwd = 32, kPassBwd = 32;  // steps of a wavefront
Form form_of(const gs_documents& d, int64_t rows, int steps) {
  const int64_t longest = d.max_q_len > 0 && d.max_q_len < rows ? d.max_q_len : rows;
  if (longest <= kChunk) return kDirectForm;
  return longest <= (int64_t)1024 * steps * kPassWaves ? kPassForm : kThreeForm;
}
uint32_t pass_chunks(int64_t rows, int32_t count, int steps) {
  return (uint32_t)(rows / (steps * kPassWaves) + count);
}
// Workspace of a form: the ticket, the maps and the states; or the chunks' maps
// and states.
size_t form_bytes(const gs_scan_config& cfg, const gs_documents& d, int64_t rows, int steps) {
  switch (form_of(d, rows, steps)) {
    case kDirectForm: return 0;
    case kPassForm:
      return 256 + (size_t)pass_chunks(rows, d.count, steps) * cfg.channels * sizeof(uint64_t) +
             (size_t)d.count * cfg.channels * sizeof(float);
    default: return (size_t)chunk_bound(rows, d.count) * cfg.channels * 2 * sizeof(float);
  }
}

GatedArgs make_args(const gs_scan_config& cfg, const gs_documents& d, int64_t rows, int V,
                   void* workspace) {
  GatedArgs a = {};
  a.docs.count = d.count;
  a.docs.rows_q = a.docs.rows_k = (int)rows;
  a.docs.q_start = d.q_start;
  a.docs.q_len = d.q_len;
  a.channels = (int)cfg.channels;
  a.groups = (a.channels + 64 * V - 1) / (64 * V);
  a.coupled = cfg.coupled;
  a.chunks = chunk_bound(rows, d.count);
  a.maps = (float*)workspace;
  a.carry = a.maps + (int64_t)a.chunks * a.channels;
  return a;
}

dim3 grid_of(const GatedArgs& a, bool direct) {
  const int64_t waves = (int64_t)(direct ? (uint32_t)a.docs.count : a.chunks) * a.groups;
  return dim3((uint32_t)((waves + 3) / 4));
}

// Long documents (a thousand chunks: 27 us with 16 lanes a channel) are shared
// among 64 lanes.
template <bool kBack>
hipError_t run_carry(GatedArgs a, hipStream_t s) {
  const int64_t blocks = (int64_t)((a.channels + 15) / 16) * a.docs.count;
  const int lanes = a.chunks / a.docs.count > 128 ? 1024 : 256;
  return launch_all(blocks, lanes, [&](uint32_t first, dim3 grid) {
    a.block0 = first;
    if (lanes == 1024) gated_carry_kernel<kBack, 64><<<grid, dim3(lanes), 0, s>>>(a);
    else gated_carry_kernel<kBack, 16><<<grid, dim3(lanes), 0, s>>>(a);
  });
}

// The one-pass form: clear, then a workgroup a chunk and channel group.
struct Pass {
  uint32_t* ticket;
  uint64_t* maps;
  uint32_t chunks;
  dim3 grid;
};
hipError_t clear_pass(GatedArgs& a, int64_t rows, int steps, int V, void* workspace, Pass& p,
                      hipStream_t s) {
  p.ticket = (uint32_t*)workspace;
  p.maps = (uint64_t*)((char*)workspace + 256);
  p.chunks = pass_chunks(rows, a.docs.count, steps);
  a.groups = (a.channels + 64 * V - 1) / (64 * V);
  p.grid = dim3(p.chunks * (uint32_t)a.groups);
  const int64_t words = (int64_t)p.chunks * a.channels;
  const int64_t work = words > (int64_t)a.docs.count * a.channels
                           ? words : (int64_t)a.docs.count * a.channels;
  const int64_t blocks = (work + 1023) / 1024;
  gated_clear_kernel<<<dim3((uint32_t)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s>>>(
      a, p.maps, words, p.ticket, (float*)(p.maps + words));
  a.state_in = (float*)(p.maps + words);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t run_fwd(GatedArgs a, Form form, int64_t rows, void* workspace, hipStream_t s) {
  const dim3 block(256);
  if (form == kPassForm) {
    Pass p;
    const hipError_t e = clear_pass(a, rows, kPassFwd, Pack<T>::V, workspace, p, s);
    if (e != hipSuccess) return e;
    gated_pass_kernel<T, kPassFwd><<<p.grid, dim3(64 * kPassWaves), 0, s>>>(a, p.maps, p.chunks,
                                                                            p.ticket);
    return hipGetLastError();
  }
  if (form == kDirectForm) {
    gated_run_kernel<T, V, true><<<grid_of(a, true), block, 0, s>>>(a);
    return hipGetLastError();
  }
  gated_maps_kernel<T, V><<<grid_of(a, false), block, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = run_carry<false>(a, s);
  if (e != hipSuccess) return e;
  gated_run_kernel<T, V, false><<<grid_of(a, false), block, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t run_bwd(GatedArgs a, Form form, int64_t rows, void* workspace, hipStream_t s) {
  const dim3 block(256);
  if (form == kPassForm) {
    Pass p;
    const hipError_t e = clear_pass(a, rows, kPassBwd, Pack<T>::V, workspace, p, s);
    if (e != hipSuccess) return e;
    gated_pass_bwd_kernel<T, kPassBwd>
        <<<p.grid, dim3(64 * kPassWaves), 0, s>>>(a, p.maps, p.chunks, p.ticket);
    return hipGetLastError();
  }
  if (form == kDirectForm) {
    gated_run_bwd_kernel<T, V, true><<<grid_of(a, true), block, 0, s>>>(a);
    return hipGetLastError();
  }
  gated_maps_bwd_kernel<T, V><<<grid_of(a, false), block, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = run_carry<true>(a, s);
  if (e != hipSuccess) return e;
  gated_run_bwd_kernel<T, V, false><<<grid_of(a, false), block, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

extern "C" {

// One size for both directions, so that a training program can keep one.
size_t gs_gated_scan_bytes(const gs_scan_config& cfg, const gs_documents& d, int64_t rows) {
  const size_t fwd = form_bytes(cfg, d, rows, kPassFwd), bwd = form_bytes(cfg, d, rows, kPassBwd);
  return fwd > bwd ? fwd : bwd;
}

// Whether the workgroups search the documents for their steps (with saved
// states they all do).
bool gs_gated_searches(const gs_documents& d, int64_t rows) {
  return form_of(d, rows, kPassFwd) != kDirectForm;
}

size_t gs_gated_saved_bytes(const gs_scan_config& cfg, const gs_documents& d, int64_t rows) {
  return (size_t)chunk_bound(rows, d.count) * (kChunk / kSub) * cfg.channels * sizeof(float);
}

hipError_t gs_launch_gated_fwd(const gs_scan_config& cfg, const gs_documents& d, int64_t rows,
                              const gs_rows& gate, const gs_rows& x, const float* state_in,
                              const gs_rows& y, float* state_out, float* saved, void* workspace,
                              hipStream_t s) {
  constexpr int V = 4;  // 8 bytes a lane of a 16-bit type, 16 of fp32
  GatedArgs a = make_args(cfg, d, rows, V, workspace);
  a.gate = gate.data; a.gate_row = gate.row;
  a.x = x.data; a.x_row = x.row;
  a.y = y.data; a.y_row = y.row;
  a.state_in = state_in;
  a.state_out = state_out;
  a.saved = saved;
  const Form form = form_of(d, rows, kPassFwd);
  if (cfg.dtype == GS_F32) return run_fwd<float, V>(a, form, rows, workspace, s);
  if (cfg.dtype == GS_BF16) return run_fwd<Bf16, V>(a, form, rows, workspace, s);
  return run_fwd<F16, V>(a, form, rows, workspace, s);
}

hipError_t gs_launch_gated_bwd(const gs_scan_config& cfg, const gs_documents& d, int64_t rows,
                              const gs_rows& gate, const gs_rows& x, const float* saved,
                              const gs_rows& dy, const float* dstate_out, const gs_rows& dgate,
                              const gs_rows& dx, float* dstate_in, void* workspace,
                              hipStream_t s) {
  constexpr int V = 2;  // 16 steps of three inputs and the states stay in registers
  GatedArgs a = make_args(cfg, d, rows, V, workspace);
  a.gate = gate.data; a.gate_row = gate.row;
  a.x = x.data; a.x_row = x.row;
  a.dy = dy.data; a.dy_row = dy.row;
  a.dgate = dgate.data; a.dgate_row = dgate.row;
  a.dx = dx.data; a.dx_row = dx.row;
  a.state_in = dstate_out;
  a.state_out = dstate_in;
  a.saved = const_cast<float*>(saved);
  const Form form = form_of(d, rows, kPassBwd);
  if (cfg.dtype == GS_F32) return run_bwd<float, V>(a, form, rows, workspace, s);
  if (cfg.dtype == GS_BF16) return run_bwd<Bf16, V>(a, form, rows, workspace, s);
  return run_bwd<F16, V>(a, form, rows, workspace, s);
}

}  // extern "C"
