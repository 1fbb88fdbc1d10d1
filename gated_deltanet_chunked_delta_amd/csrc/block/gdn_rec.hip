// gdn_rec.hip -- gated linear recurrence, channels last, its gradient, its single token.
//
//   a_t = exp(L_t),  L = g  or  -scale sigmoid(g),  m = 1  or  sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t s_t x_t,   s = 1 or sigmoid(i)
//   dh_t = dy_t + a_{t+1} dh_{t+1}
//   dx = dh m s,  di = dh m x s (1 - s),
//   dL = a dh h_{t-1} - [with scale] dh s x a^2 / m,   dg = dL  or  -dL scale sigmoid'(g)
//
// Bound: memory, with nearly as much arithmetic (some 60 instructions an element, four
// or five of them transcendental).  So every input is read once and every gate formed
// once: a workgroup takes a chunk of tokens of 64 lanes' channels, a wave to every S
// tokens, and holds decays and inputs in registers while it waits for the state that
// enters its chunk.  All sequences of a call lie along one axis of tokens, whatever their
// lengths.  What a chunk (or a wave's part) makes of the state entering it is one pair per
// channel, (A, U): A h + U -- or U alone where a sequence starts inside, marked by A = -1
// (a product of decays is never negative), so that a value that is not finite reaches no
// other sequence.
//
// Chunks hand their pairs on through global words of 64 bits, written and read whole by
// relaxed atomics past the dies' caches; a word of zeros is not written yet.  Chunks lie
// in groups: a chunk composes the pairs of its group's chunks before it, in order, and
// applies them to the state that leaves the group before, which that group's last chunk
// writes.  Which words are read does not depend on time, so results do not either.  Every
// wait ends: workgroups of the same channels number themselves by a counter when they
// start, and wait only for words of lower numbers, whose workgroups run already and wait for
// none above theirs.
// The gradient's chain runs the other way with pairs of its own: in token order its U is
// the sum of dy_t times the decays up to t, cut off at the first sequence's end.
//
// Measured (bf16, scale and i): 65,536 tokens of 2,048 channels in 299-320 us (1.07 GB, 3.6-3.4
// TB/s; three kernels that read the inputs twice: 950), its gradient in 545-556 (1.88 GB, 3.4
// TB/s); 16,384 of 2,304 in 87-93 and 150-156 us.  fp32, one channel a thread: 420 and 752 us (2.15
// and 3.76 GB, 5.1 and 5.0 TB/s), 16,384 of 2,304 121 and 218.  Four bytes of a row a thread and 16
// (gradient: 8) tokens, eight waves (groups of 16 in all of these: 326, 580): with eight bytes and
// half the tokens 413 and 1,075 us (the gradient's registers spill); 8 tokens forwards 342; the
// gradient with 4 tokens 792, with chunks of four or two waves 611 and 801.  A gradient that
// keeps its inputs' products too spills: 697.
#include "gdn_block.h"

namespace gdn {

namespace {

template <class E> constexpr int kRV = REC_BYTES / (int)sizeof(E);  // channels of a thread

// The sequence of a token, among the non-empty ones.
struct RecSeq {
  const int32_t* cu;
  int N, T, tokens;
  int n, start, end;  // clamped to [0, tokens]: a bad device copy of cu reads nothing out of bounds
  __device__ __forceinline__ explicit RecSeq(const RecParams& p)
      : cu(p.cu), N(p.N), T(p.T), tokens(p.tokens), n(0), start(0), end(0) {}
  __device__ __forceinline__ void bounds() {
    if (cu) {
      start = min(max(cu[n], 0), tokens);
      end = min(max(cu[n + 1], 0), tokens);
    } else {
      start = n * T;
      end = start + T;
    }
  }
  // past the last token of any sequence
  __device__ __forceinline__ int all() const { return cu ? min(max(cu[N], 0), tokens) : tokens; }
  __device__ __forceinline__ bool seek(int t) {
    if (cu) {
      int lo = 0, hi = N - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      n = lo;
    } else {
      n = t / T;
    }
    bounds();
    return t >= start && t < end;
  }
  // to the sequence that starts where this one ended; false behind the last
  __device__ __forceinline__ bool next() {
    const int t = end;
    do {
      if (++n >= N) return false;
      bounds();
    } while (end <= start);
    return start == t;
  }
};

// exp(L) - 1 for L <= 0 within a few roundings of its value: the series near 0 (the
// first term left out is below 2^-25 of the sum), the difference elsewhere.
__device__ __forceinline__ float expm1_neg(float L, float a) {
  float s = fmaf(L, 1.f / 120, 1.f / 24);
  s = fmaf(L, s, 1.f / 6);
  s = fmaf(L, s, 0.5f);
  s = fmaf(L, s, 1.f) * L;
  return L > -0.1f ? s : a - 1.f;
}

// (The fp32 gate holds its argument to a range, a NaN too: here it stays one.)
template <class E>
__device__ __forceinline__ float rec_sigmoid(float x) {
  const float s = fast_sigmoid<E>(x);
  return sizeof(E) == 4 && x != x ? x : s;
}

// Decay, input and what the gradient needs of them, of one token and channel.
template <class E, class GT, bool SC, bool IN>
struct RecGate {
  float a, u, sg, m, si;
  __device__ __forceinline__ RecGate(float x, float g, float i, float scale) {
    float L = g;
    if (SC) {
      sg = rec_sigmoid<GT>(g);
      L = -scale * sg;
    }
    a = __builtin_amdgcn_exp2f(1.44269504f * L);
    m = si = 1.f;
    u = x;
    if (SC) {  // 1 - a^2 without the cancellation where a is near 1
      const float e = expm1_neg(L, a);
      m = __builtin_amdgcn_sqrtf(fmaf(-e, e, -2.f * e));
      u *= m;
    }
    if (IN) {
      si = rec_sigmoid<E>(i);
      u *= si;
    }
  }
};

// The V channels of a thread's token, as loaded: unpacked where they are used, so that
// many loads are under way at once.  A row's last thread may have fewer than V channels
// left: it loads the row's last V (D >= V) and finds its own `shift` elements on.
template <class E, int V>
struct RecRaw {
  typedef E vec __attribute__((ext_vector_type(V)));
  vec t;
  __device__ __forceinline__ void load(const E* p, int shift) {
    typedef vec any __attribute__((aligned(sizeof(E))));
    t = *reinterpret_cast<const any*>(p - shift);
  }
  __device__ __forceinline__ float get(int e, int shift) const {
    float f = to_f(t[e]);
#pragma unroll
    for (int s = 1; s < V; ++s)
      if (e + s < V) f = shift == s ? to_f(t[e + s]) : f;
    return f;
  }
};
template <> struct RecRaw<bf16, 1> {
  bf16 t;
  __device__ __forceinline__ void load(const bf16* p, int) { t = *p; }
  __device__ __forceinline__ float get(int, int) const { return to_f(t); }
};
template <> struct RecRaw<float, 1> {
  float t;
  __device__ __forceinline__ void load(const float* p, int) { t = *p; }
  __device__ __forceinline__ float get(int, int) const { return t; }
};
// (Past the L2: 16,384 tokens of 2,048 channels 83 and 142 us, 87 and 151 with ordinary stores.)
template <int V, class E>
__device__ __forceinline__ void rec_st(E* p, int n, const float (&f)[V]) {
  typedef E vec __attribute__((ext_vector_type(V)));
  typedef vec any __attribute__((aligned(sizeof(E))));
  if (n >= V) {
    vec t;
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = to_e<E>(f[e]);
    __builtin_nontemporal_store(t, reinterpret_cast<any*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < n) p[e] = to_e<E>(f[e]);
  }
}

// Blocks are numbered channels first over the chunks: neighbours read neighbouring lines.
// (Fewer than 2^32: 2^40 entries of at least 2,048 a block, or 2^25 chunks.)
__device__ __forceinline__ uint32_t rec_block() { return (uint32_t)block_2d(); }
template <int V> __host__ __device__ __forceinline__ uint32_t rec_width(int D) { return ((uint32_t)D + 64 * V - 1) / (64 * V); }
template <int V>
__device__ __forceinline__ void rec_vec(const float* base, int64_t row, int D, int c, int n, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = base && e < n ? base[row * D + c + e] : 0.f;
}
template <int V>
__device__ __forceinline__ void rec_put(float* base, int64_t row, int D, int c, int n, const float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < n) base[row * D + c + e] = f[e];
}

__device__ __forceinline__ float rec_apply(float2 s, float h) { return s.x < 0.f ? s.y : fmaf(s.x, h, s.y); }
// first r, then v
__device__ __forceinline__ float2 rec_then(float2 r, float2 v) {
  return v.x < 0.f ? v : make_float2(r.x < 0.f ? -1.f : r.x * v.x, fmaf(v.x, r.y, v.y));
}

// ---------------------------------------------------------------- the chunks' chain
// A pair as a word that is never 0 (the first half inverted: 0 would be a NaN of all ones,
// which NaNs are replaced by another for).
__device__ __forceinline__ uint64_t rec_word(float2 v) {
  const uint32_t a = v.x != v.x ? 0x7fc00000u : __builtin_bit_cast(uint32_t, v.x);
  return (uint64_t)~a << 32 | __builtin_bit_cast(uint32_t, v.y);
}
__device__ __forceinline__ float2 rec_pair(uint64_t w) {
  return make_float2(__builtin_bit_cast(float, ~(uint32_t)(w >> 32)), __builtin_bit_cast(float, (uint32_t)w));
}
__device__ __forceinline__ void rec_publish(uint64_t* p, float2 v) {
  __hip_atomic_store(p, rec_word(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t rec_peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t rec_await(const uint64_t* p) {
  uint64_t w = rec_peek(p);
  while (w == 0) {
    __builtin_amdgcn_s_sleep(1);
    w = rec_peek(p);
  }
  return w;
}
// Words in front of the chunks': a counter for each workgroup's width of channels (the
// narrowest, fp32's), each in a line of its own.
constexpr int REC_LINE = 16;
__host__ __device__ __forceinline__ int64_t rec_counters(int D) { return (int64_t)rec_width<REC_BYTES / 4>(D) * REC_LINE; }
// Chunks of a group.  Groups wait for each other, some 1.2 us a time; a chunk reads half a
// group's words.  Many channels bring enough other workgroups for the first and pay for the
// second.  Measured with 8, 16, 32 chunks (65,536 tokens, forward and gradient): 2,048 channels
// 320 + 551, 329 + 569, 353 + 604 us; 512 88 + 153, 88 + 152, 94 + 164; 128 59 + 94, 46 + 65, 41 + 60.
constexpr int REC_GROUP_MIN = 8;
template <int V> __device__ __forceinline__ int rec_group(int D) { return rec_width<V>(D) >= 8 ? REC_GROUP_MIN : 16; }
constexpr int REC_PEEK = 4;    // words requested together

// Publishes the pair of chunk k (counted in the chain's direction) and returns the state
// entering it.  One wave; e: the thread's channel, of which all V exist up to n.
template <int V>
__device__ __forceinline__ void rec_chain(const RecParams& p, int k, int c, int n, const float2 (&own)[V], float (&h)[V]) {
  const int len = rec_group<V>(p.D), group = k / len, first = group * len;
  uint64_t* pairs = p.words + rec_counters(p.D);          // [nchunk][D]
  uint64_t* ends = pairs + (int64_t)p.nchunk * p.D;       // [groups][D]: (-1, the state leaving a group)
  const bool last = k == first + len - 1;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < n && !last) rec_publish(pairs + (int64_t)k * p.D + c + e, own[e]);
  float2 r[V];
#pragma unroll
  for (int e = 0; e < V; ++e) r[e] = make_float2(1.f, 0.f);
  for (int j = first; j < k; j += REC_PEEK) {
    uint64_t w[REC_PEEK][V];
#pragma unroll
    for (int q = 0; q < REC_PEEK; ++q)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (j + q < k && e < n) w[q][e] = rec_peek(pairs + (int64_t)(j + q) * p.D + c + e);
#pragma unroll
    for (int q = 0; q < REC_PEEK; ++q)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (j + q < k && e < n) {
          if (w[q][e] == 0) w[q][e] = rec_await(pairs + (int64_t)(j + q) * p.D + c + e);
          r[e] = rec_then(r[e], rec_pair(w[q][e]));
        }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float in = 0.f;
    if (first > 0 && e < n) in = rec_pair(rec_await(ends + (int64_t)(group - 1) * p.D + c + e)).y;
    h[e] = rec_apply(r[e], in);
    if (e < n && last) rec_publish(ends + (int64_t)group * p.D + c + e, make_float2(-1.f, rec_apply(own[e], h[e])));
  }
}

// The chunk of this workgroup, counted in the chain's direction: its own number where it
// waits for nobody, else by its channels' counter.
template <int V>
__device__ __forceinline__ int rec_ticket(const RecParams& p) {
  const uint32_t wide = rec_width<V>(p.D), own = rec_block() / wide;
  if (!p.words || own >= (uint32_t)p.nchunk) return (int)own;
  __shared__ uint32_t id;
  if (threadIdx.x == 0)
    id = __hip_atomic_fetch_add(reinterpret_cast<uint32_t*>(p.words + rec_block() % wide * REC_LINE), 1u, __ATOMIC_RELAXED,
                                __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return (int)__builtin_amdgcn_readfirstlane(id);
}

// Where sequences start and end among the tokens [t0, t0 + S) of a wave: bit k, token t0 +
// k.  `count` tokens from t0 on belong to sequences; none do behind them.
template <int S>
struct RecSpan {
  uint32_t starts = 0, ends = 0;
  int count = 0;
  __device__ __forceinline__ RecSpan(const RecParams& p, int t0, int t1) {
    RecSeq s(p);
    t1 = min(t1, s.all());
    if (t0 >= t1 || !s.seek(t0)) return;
    if (s.start == t0) starts = 1;
    count = t1 - t0;
    while (s.end <= t1) {
      ends |= 1u << (s.end - 1 - t0);
      if (s.end == t1) break;
      if (!s.next()) {
        count = s.end - t0;  // (a bad device copy of cu: a gap)
        break;
      }
      starts |= 1u << (s.start - t0);
    }
  }
};
// The sequence of token t.
__device__ __forceinline__ int rec_seq_of(const RecParams& p, int t) {
  RecSeq s(p);
  s.seek(t);
  return s.n;
}
template <int V>
__device__ __forceinline__ void rec_state(const RecParams& p, const float* states, int t, int c, int n, float (&h)[V]) {
  rec_vec<V>(states, states ? rec_seq_of(p, t) : 0, p.D, c, n, h);
}

// Workgroups past the chunks write the final states of sequences without tokens, each
// looking at REC_EMPTY of them.
constexpr int REC_EMPTY = 64;
template <int V>
__device__ __forceinline__ void rec_empty_seqs(const RecParams& p, int group, const float* src, float* dst, int c, int n) {
  if (n <= 0) return;
  RecSeq s(p);
  for (int q = group * REC_EMPTY + wave_id(); q < min((group + 1) * REC_EMPTY, p.N); q += REC_W) {
    s.n = q;
    s.bounds();
    if (s.end > s.start) continue;
    float h[V];
    rec_vec<V>(src, q, p.D, c, n, h);
    rec_put<V>(dst, q, p.D, c, n, h);
  }
}

template <class E, class GT, int V, bool SC, bool IN>
__global__ __launch_bounds__(64 * REC_W, 4) void rec_fwd_kernel(RecParams p) {
  constexpr int S = REC_FS, W = REC_W;
  __shared__ float2 pairs[W][64 * V];
  __shared__ float entering[64 * V];
  const int ch = rec_ticket<V>(p);
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
  const int c = (int)(rec_block() % rec_width<V>(p.D) * 64 + lane) * V, n = p.D - c, shift = max(V - n, 0);
  if (ch >= p.nchunk) {
    rec_empty_seqs<V>(p, ch - p.nchunk, p.h0, p.hT, c, n);
    return;
  }
  const int t0 = ch * (W * S) + w * S;
  const RecSpan<S> span(p, t0, min(t0 + S, p.tokens));
  float a[S][V], u[S][V], scale[V];
  float2 f[V];
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = make_float2(1.f, 0.f);
  if (n > 0 && span.count) {
    RecRaw<E, V> x[S], i[S];
    RecRaw<GT, V> g[S];
    rec_vec<V>(p.scale, 0, p.D, c, n, scale);
    const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c;
    const GT* gp = static_cast<const GT*>(p.g) + t0 * p.g_stride + c;
    const E* ip = static_cast<const E*>(p.i) + (IN ? t0 * p.i_stride + c : 0);
#pragma unroll
    for (int k = 0; k < S; ++k) {  // (behind the last token: that one again)
      const int t = min(k, span.count - 1);
      g[k].load(gp + t * p.g_stride, shift);
      x[k].load(xp + t * p.x_stride, shift);
      if (IN) i[k].load(ip + t * p.i_stride, shift);
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k < span.count) {
        if (span.starts >> k & 1) {
          float t[V];
          rec_state<V>(p, p.h0, t0 + k, c, n, t);
#pragma unroll
          for (int e = 0; e < V; ++e) f[e].y = t[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const RecGate<E, GT, SC, IN> q(x[k].get(e, shift), g[k].get(e, shift), IN ? i[k].get(e, shift) : 0.f, scale[e]);
          a[k][e] = q.a;
          u[k][e] = q.u;
          f[e] = make_float2(f[e].x * q.a, fmaf(q.a, f[e].y, q.u));
        }
      }
    }
    if (span.starts) {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e].x = -1.f;
    }
  }
  if (n > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) pairs[w][lane * V + e] = f[e];
  }
  __syncthreads();
  if (p.words) {
    if (w == 0 && n > 0) {
      float2 own[V];
      float h[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        own[e] = pairs[0][lane * V + e];
#pragma unroll
        for (int q = 1; q < W; ++q) own[e] = rec_then(own[e], pairs[q][lane * V + e]);
      }
      rec_chain<V>(p, ch, c, n, own, h);
#pragma unroll
      for (int e = 0; e < V; ++e) entering[lane * V + e] = h[e];
    }
    __syncthreads();
  }
  if (n <= 0) return;
  float h[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    h[e] = p.words ? entering[lane * V + e] : 0.f;
    for (int q = 0; q < w; ++q) h[e] = rec_apply(pairs[q][lane * V + e], h[e]);
  }
  if (p.enter && w % (REC_STATE / S) == 0 && t0 < p.tokens) rec_put<V>(p.enter, t0 / REC_STATE, p.D, c, n, h);
  E* yp = static_cast<E*>(p.y) + (int64_t)t0 * p.D + c;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if (k < span.count) {
      if (span.starts >> k & 1) rec_state<V>(p, p.h0, t0 + k, c, n, h);
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = fmaf(a[k][e], h[e], u[k][e]);
      if (p.y) rec_st<V>(yp + (int64_t)k * p.D, n, h);
      if ((span.ends >> k & 1) && p.hT) rec_put<V>(p.hT, rec_seq_of(p, t0 + k), p.D, c, n, h);
    }
  }
}

// Gradient.  The first walk forms the gates and the waves' pairs of both chains; while one
// wave waits for the carry from behind, the others walk forward from the state entering
// the chunk (kept by the forward pass) to the states before every token; then back.
template <class E, class GT, int V, bool SC, bool IN>
__global__ __launch_bounds__(64 * REC_W, 4) void rec_bwd_kernel(RecParams p) {
  constexpr int S = REC_BS, W = REC_W;
  __shared__ float2 fw[W][64 * V], bw[W][64 * V];
  __shared__ float leaving[64 * V];
  const int k_chain = rec_ticket<V>(p);
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
  const int c = (int)(rec_block() % rec_width<V>(p.D) * 64 + lane) * V, n = p.D - c, shift = max(V - n, 0);
  if (k_chain >= p.nchunk) {
    rec_empty_seqs<V>(p, k_chain - p.nchunk, p.dhT, p.dh0, c, n);
    return;
  }
  const int ch = p.nchunk - 1 - k_chain, t0 = ch * (W * S) + w * S;
  const RecSpan<S> span(p, t0, min(t0 + S, p.tokens));
  RecRaw<E, V> x[S], dy[S];
  float a[S][V], m[S][V], sg[S][V], si[S][V], h[S][V], scale[V];
  float2 f[V], b[V];
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = b[e] = make_float2(1.f, 0.f);
  const bool live = n > 0 && span.count;
  if (live) {
    RecRaw<E, V> i[S];
    RecRaw<GT, V> g[S];
    rec_vec<V>(p.scale, 0, p.D, c, n, scale);
    const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c;
    const GT* gp = static_cast<const GT*>(p.g) + t0 * p.g_stride + c;
    const E* ip = static_cast<const E*>(p.i) + (IN ? t0 * p.i_stride + c : 0);
    const E* dp = static_cast<const E*>(p.dy) + (int64_t)t0 * p.D + c;
#pragma unroll
    for (int k = 0; k < S; ++k) {  // (behind the last token: that one again)
      const int t = min(k, span.count - 1);
      g[k].load(gp + t * p.g_stride, shift);
      x[k].load(xp + t * p.x_stride, shift);
      if (IN) i[k].load(ip + t * p.i_stride, shift);
      dy[k].load(dp + (int64_t)t * p.D, shift);
    }
    bool cut = false;  // behind the first sequence's end nothing more reaches the front
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k < span.count) {
        if (span.starts >> k & 1) {
          float t[V];
          rec_state<V>(p, p.h0, t0 + k, c, n, t);
#pragma unroll
          for (int e = 0; e < V; ++e) f[e].y = t[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const RecGate<E, GT, SC, IN> q(x[k].get(e, shift), g[k].get(e, shift), IN ? i[k].get(e, shift) : 0.f, scale[e]);
          a[k][e] = q.a;
          if (SC) { m[k][e] = q.m; sg[k][e] = q.sg; }
          if (IN) si[k][e] = q.si;
          f[e] = make_float2(f[e].x * q.a, fmaf(q.a, f[e].y, q.u));
          if (!cut) b[e] = make_float2(b[e].x * q.a, fmaf(b[e].x * q.a, dy[k].get(e, shift), b[e].y));
        }
        if ((span.ends >> k & 1) && !cut) {
          cut = true;
          float t[V];
          rec_state<V>(p, p.dhT, t0 + k, c, n, t);
#pragma unroll
          for (int e = 0; e < V; ++e) b[e].y = fmaf(b[e].x, t[e], b[e].y);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (span.starts) f[e].x = -1.f;
      if (cut) b[e].x = -1.f;
    }
  }
  if (n > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      fw[w][lane * V + e] = f[e];
      bw[w][lane * V + e] = b[e];
    }
  }
  __syncthreads();
  if (p.words && w == 0 && n > 0) {
    float2 own[V];
    float d[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      own[e] = bw[W - 1][lane * V + e];
#pragma unroll
      for (int q = W - 2; q >= 0; --q) own[e] = rec_then(own[e], bw[q][lane * V + e]);
    }
    rec_chain<V>(p, k_chain, c, n, own, d);
#pragma unroll
    for (int e = 0; e < V; ++e) leaving[lane * V + e] = d[e];
  }
  if (live) {  // the states before every token
    float hc[V];
    rec_vec<V>(p.enter, ch, p.D, c, n, hc);
#pragma unroll
    for (int e = 0; e < V; ++e)
      for (int q = 0; q < w; ++q) hc[e] = rec_apply(fw[q][lane * V + e], hc[e]);
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k < span.count) {
        if (span.starts >> k & 1) rec_state<V>(p, p.h0, t0 + k, c, n, hc);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float u = x[k].get(e, shift);  // (formed again: the products of the gate, in its order)
          if (SC) u *= m[k][e];
          if (IN) u *= si[k][e];
          h[k][e] = hc[e];
          hc[e] = fmaf(a[k][e], hc[e], u);
        }
      }
    }
  }
  __syncthreads();
  float ds[V] = {};
  if (live) {
    float dc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      dc[e] = p.words ? leaving[lane * V + e] : 0.f;
      for (int q = W - 1; q > w; --q) dc[e] = rec_apply(bw[q][lane * V + e], dc[e]);
    }
    E* dxp = static_cast<E*>(p.dx) + (int64_t)t0 * p.D + c;
    GT* dgp = static_cast<GT*>(p.dg) + (int64_t)t0 * p.D + c;
    E* dip = static_cast<E*>(p.di) + (IN ? (int64_t)t0 * p.D + c : 0);
#pragma unroll
    for (int k = S - 1; k >= 0; --k) {
      if (k < span.count) {
        if (span.ends >> k & 1) rec_state<V>(p, p.dhT, t0 + k, c, n, dc);
        float dx[V], dg[V], di[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xv = x[k].get(e, shift), dh = dy[k].get(e, shift) + dc[e], dhs = IN ? dh * si[k][e] : dh;
          dc[e] = a[k][e] * dh;
          dx[e] = SC ? dhs * m[k][e] : dhs;
          if (IN) di[e] = dx[e] * xv * (1.f - si[k][e]);
          float dl = dc[e] * h[k][e];
          if (SC) {
            const float im = m[k][e] == 0.f ? 0.f : __builtin_amdgcn_rcpf(m[k][e]);
            dl -= dhs * xv * (a[k][e] * a[k][e]) * im;
            dg[e] = -dl * scale[e] * (sg[k][e] - sg[k][e] * sg[k][e]);
            ds[e] -= dl * sg[k][e];
          } else {
            dg[e] = dl;
          }
        }
        rec_st<V>(dxp + (int64_t)k * p.D, n, dx);
        rec_st<V>(dgp + (int64_t)k * p.D, n, dg);
        if (IN) rec_st<V>(dip + (int64_t)k * p.D, n, di);
        if ((span.starts >> k & 1) && p.dh0) rec_put<V>(p.dh0, rec_seq_of(p, t0 + k), p.D, c, n, dc);
      }
    }
  }
  if (!SC) return;
  if (n > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) fw[w][lane * V + e].x = ds[e];  // (last read before the barrier above)
  }
  __syncthreads();
  if (w == 0 && n > 0) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) t += fw[q][lane * V + e].x;
      ds[e] = t;
    }
    rec_put<V>(p.part, ch, p.D, c, n, ds);
  }
}

// Zeros: words that are not written yet, and the counter.
__global__ __launch_bounds__(256) void rec_clear_kernel(uint64_t* p, int64_t words) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < words; i += gridDim.x * 256ll) p[i] = 0;
}

template <class E, class GT, int V, bool SC, bool IN>
__global__ __launch_bounds__(64) void rec_step_kernel(RecStepParams p) {
  const uint32_t wide = rec_width<V>(p.D);
  const int c = (int)(blockIdx.x % wide * 64 + threadIdx.x) * V, n = p.D - c, r = (int)(blockIdx.x / wide), shift = max(V - n, 0);
  if (n <= 0) return;
  const int slot = p.state_idx ? p.state_idx[r] : r;
  if (slot < 0 || slot >= p.num_slots) return;
  RecRaw<E, V> x, i;
  RecRaw<GT, V> g;
  x.load(static_cast<const E*>(p.x) + r * p.x_stride + c, shift);
  g.load(static_cast<const GT*>(p.g) + r * p.g_stride + c, shift);
  if (IN) i.load(static_cast<const E*>(p.i) + r * p.i_stride + c, shift);
  float h[V], scale[V];
  rec_vec<V>(p.state, slot, p.D, c, n, h);
  rec_vec<V>(p.scale, 0, p.D, c, n, scale);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const RecGate<E, GT, SC, IN> w(x.get(e, shift), g.get(e, shift), IN ? i.get(e, shift) : 0.f, scale[e]);
    h[e] = fmaf(w.a, h[e], w.u);
  }
  rec_put<V>(p.state, slot, p.D, c, n, h);
  rec_st<V>(static_cast<E*>(p.y) + (int64_t)r * p.D + c, n, h);
}

// f<E, GT, V, SC, IN>() by the call's types and optional inputs; rows of fewer channels
// than a thread takes go one by one.
template <class E, class GT, int V, class F>
void rec_pick(bool sc, bool in, F f) {
  if (sc && in) f.template operator()<E, GT, V, true, true>();
  else if (sc) f.template operator()<E, GT, V, true, false>();
  else if (in) f.template operator()<E, GT, V, false, true>();
  else f.template operator()<E, GT, V, false, false>();
}
template <class E, class GT, class F>
void rec_width_of(int D, bool sc, bool in, F f) {
  if constexpr (kRV<E> > 1)
    if (D < kRV<E>) return rec_pick<E, GT, 1>(sc, in, f);
  rec_pick<E, GT, kRV<E>>(sc, in, f);
}
template <class F>
hipError_t rec_types(int dtype, int g_f32, int D, bool sc, bool in, F f) {
  if (dtype == GDN_F32) rec_width_of<float, float>(D, sc, in, f);
  else if (g_f32) rec_width_of<bf16, float>(D, sc, in, f);
  else rec_width_of<bf16, bf16>(D, sc, in, f);
  return hipGetLastError();
}
struct RecLaunch {
  bool bwd;
  const RecParams& p;
  hipStream_t st;
  template <class E, class GT, int V, bool SC, bool IN>
  void operator()() const {
    // (sequences of one length are empty all or none)
    const int more = (bwd ? p.dh0 : p.hT) && (p.cu || p.tokens == 0) ? (p.N + REC_EMPTY - 1) / REC_EMPTY : 0;
    if (p.nchunk + more == 0) return;
    const dim3 grid = blocks_2d(rec_width<V>(p.D) * (int64_t)(p.nchunk + more));
    if (bwd) hipLaunchKernelGGL((rec_bwd_kernel<E, GT, V, SC, IN>), grid, dim3(64 * REC_W), 0, st, p);
    else hipLaunchKernelGGL((rec_fwd_kernel<E, GT, V, SC, IN>), grid, dim3(64 * REC_W), 0, st, p);
  }
};
struct RecStepLaunch {
  const RecStepParams& p;
  hipStream_t st;
  template <class E, class GT, int V, bool SC, bool IN>
  void operator()() const {
    const dim3 grid(rec_width<V>(p.D) * (uint32_t)p.N);
    hipLaunchKernelGGL((rec_step_kernel<E, GT, V, SC, IN>), grid, dim3(64), 0, st, p);
  }
};

}  // namespace

int64_t rec_words(int nchunk, int D) { return rec_counters(D) + ((int64_t)nchunk + nchunk / REC_GROUP_MIN) * D; }
static hipError_t rec_run(int dtype, const RecParams& p, bool bwd, hipStream_t st) {
  if (p.words) {
    const int64_t n = rec_words(p.nchunk, p.D);
    hipLaunchKernelGGL(rec_clear_kernel, dim3((uint32_t)std::min<int64_t>((n + 1023) / 1024, 1024)), dim3(256), 0, st, p.words, n);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return rec_types(dtype, p.g_f32, p.D, p.scale, p.i, RecLaunch{bwd, p, st});
}
hipError_t launch_rec_fwd(int dtype, const RecParams& p, hipStream_t st) { return rec_run(dtype, p, false, st); }
hipError_t launch_rec_bwd(int dtype, const RecParams& p, hipStream_t st) { return rec_run(dtype, p, true, st); }
hipError_t launch_rec_step(int dtype, const RecStepParams& p, hipStream_t st) {
  return rec_types(dtype, p.g_f32, p.D, p.scale, p.i, RecStepLaunch{p, st});
}

}  // namespace gdn
