// gated.hip — gated linear recurrence over documents, and its gradient.
//
//   a = sigmoid(gate),  h_t = a_t h_{t-1} + u_t,
//   u_t = (1 - a_t) x_t (coupled: the over operator with alpha = 1 - a) or x_t.
//
// Backward, from the last step: g_t = dy_t + a_{t+1} g_{t+1};
//   dx = (1 - a) g or g,  dgate = g (h_{t-1} - x_t) a (1 - a) or
//   g h_{t-1} a (1 - a);  the first step sends a g to the state it took in.
//
// A step costs a dozen operations on six to twelve bytes, so the operator is
// bound by memory traffic; what stands in the way is that the steps depend on
// each other.  The recurrence is a composition of maps h -> A h + H, which is
// associative, so each document is cut into chunks of 64 steps:
//   1. every chunk composes its own map (A, H), all chunks at once;
//   2. per document and channel, the chunks' maps are applied in order to the
//      document's state: the state each chunk starts from;
//   3. every chunk runs its steps from that state and writes its outputs.
// Documents of at most a chunk need only the third, in one launch.  The order
// of every sum is fixed, so results are the same bits every time.
// Lanes run over channels, a wavefront over the steps of one chunk; states are
// fp32 throughout, and only the outputs are rounded, once.
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
};

// a = sigmoid(f) and z = 1 - a, both accurate relative to themselves (a gate
// that is nearly open has a tiny z, a shut one a tiny a).  fp32 inputs carry
// the exponent's rounding along.
template <bool kExact>
__device__ inline void gate_of(float f, float& a, float& z) {
  const float v = fabsf(f) > 128.0f ? 128.0f : fabsf(f);  // keeps NaN
  const float t = -v * kLog2e;
  float m = __builtin_amdgcn_exp2f(t);
  if constexpr (kExact) m = fmaf(m, fmaf(-v, kLog2e, -t) * kLn2, m);
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
  const int doc = blockIdx.x / per;
  const int c = threadIdx.x & 15, seg = threadIdx.x >> 4;
  const int ch = (blockIdx.x % per) * 16 + c;
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

}  // namespace gs

using namespace gs;

namespace {

uint32_t chunk_bound(int64_t rows, int32_t count) {
  return (uint32_t)(rows / kChunk + count);
}

// The one-launch form: no document is longer than a chunk.
bool direct_form(const gs_documents& d, int64_t rows) {
  const int64_t longest = d.max_q_len > 0 && d.max_q_len < rows ? d.max_q_len : rows;
  return longest <= kChunk;
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
hipError_t run_carry(const GatedArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)((a.channels + 15) / 16) * a.docs.count));
  if (a.chunks / a.docs.count > 128)
    gated_carry_kernel<kBack, 64><<<grid, dim3(1024), 0, s>>>(a);
  else
    gated_carry_kernel<kBack, 16><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t run_fwd(const GatedArgs& a, bool direct, hipStream_t s) {
  const dim3 block(256);
  if (direct) {
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
hipError_t run_bwd(const GatedArgs& a, bool direct, hipStream_t s) {
  const dim3 block(256);
  if (direct) {
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

size_t gs_gated_scan_bytes(const gs_scan_config& cfg, const gs_documents& d, int64_t rows) {
  if (direct_form(d, rows)) return 0;
  return (size_t)chunk_bound(rows, d.count) * cfg.channels * 2 * sizeof(float);
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
  const bool direct = direct_form(d, rows);
  if (cfg.dtype == GS_F32) return run_fwd<float, V>(a, direct, s);
  if (cfg.dtype == GS_BF16) return run_fwd<Bf16, V>(a, direct, s);
  return run_fwd<F16, V>(a, direct, s);
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
  const bool direct = direct_form(d, rows);
  if (cfg.dtype == GS_F32) return run_bwd<float, V>(a, direct, s);
  if (cfg.dtype == GS_BF16) return run_bwd<Bf16, V>(a, direct, s);
  return run_bwd<F16, V>(a, direct, s);
}

}  // extern "C"
