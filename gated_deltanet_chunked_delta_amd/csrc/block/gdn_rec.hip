// gdn_rec.hip -- gated linear recurrence, channels last, its gradient, its single token.
//
//   a_t = exp(L_t),  L = g  or  -scale sigmoid(g),  m = 1  or  sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t s_t x_t,   s = 1 or sigmoid(i)
//   dh_t = dy_t + a_{t+1} dh_{t+1}
//   dx = dh m s,  di = dh m x s (1 - s),
//   dL = a dh h_{t-1} - [with scale] dh s x a^2 / m,   dg = dL  or  -dL scale sigmoid'(g)
//
// Bound: memory.  All sequences of a call lie along one axis of tokens, which is cut
// into chunks whatever the sequences' lengths.  What a chunk makes of the state that
// enters it is one pair per channel, (A, U): A h + U -- or U alone where a sequence
// starts inside, marked by A = -1 (a product of decays is never negative), so that a
// value that is not finite reaches no other sequence.  One kernel forms the pairs, one
// joins them to the states entering the chunks, one walks every chunk again from there.
// The gradient's chain runs the other way with pairs of its own: in token order its
// U is the sum of dy_t times the decays up to t, cut off at the first sequence's end.
#include "gdn_block.h"

namespace gdn {

namespace {

template <class E> constexpr int kRV = 4 / (int)sizeof(E);  // channels of a thread: 4 bytes a token

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

// exp(L) - 1 for L <= 0 within two roundings of its value: the series near 0 (the
// first term left out is below 2^-25 of the sum), the difference elsewhere.
__device__ __forceinline__ float expm1_neg(float L, float a) {
  float s = fmaf(L, 1.f / 5040, 1.f / 720);
  s = fmaf(L, s, 1.f / 120);
  s = fmaf(L, s, 1.f / 24);
  s = fmaf(L, s, 1.f / 6);
  s = fmaf(L, s, 0.5f);
  s = fmaf(L, s, 1.f) * L;
  return L > -0.35f ? s : a - 1.f;
}

// Decay and input of one token and channel.
template <bool SC, bool IN>
struct RecGate {
  float a, u, sg, m, im, si;  // im = 1 / m, 0 where m is
  __device__ __forceinline__ RecGate(float x, float g, float i, float scale) {
    float L = g;
    if (SC) {
      sg = fast_sigmoid<float>(g);
      L = -scale * sg;
    }
    a = __builtin_amdgcn_exp2f(1.44269504f * L);
    m = im = si = 1.f;
    if (SC) {
      const float e = expm1_neg(L, a), m2 = -e * (2.f + e);
      const float r = __builtin_amdgcn_rsqf(m2);
      im = m2 == 0.f ? 0.f : r;
      m = m2 == 0.f ? 0.f : m2 * r;
    }
    if (IN) si = fast_sigmoid<float>(i);
    u = x;
    if (SC) u *= m;
    if (IN) u *= si;
  }
};

// The V channels at c of a token's row, as loaded; n of them exist.
template <class E, int V> struct RecRaw { E v[V]; };
template <int V, class E>
__device__ __forceinline__ void rec_ld(const E* p, int n, RecRaw<E, V>& r) {
  if (V == 2 && n >= 2) {
    if constexpr (V == 2 && sizeof(E) == 2) {
      const bf16x2 t = *reinterpret_cast<const bf16x2_any*>(p);
      r.v[0] = t[0]; r.v[1] = t[1];
    } else if constexpr (V == 2) {
      const f32x2 t = *reinterpret_cast<const f32x2_any*>(p);
      r.v[0] = t[0]; r.v[1] = t[1];
    }
  } else {
    r.v[0] = p[0];
#pragma unroll
    for (int e = 1; e < V; ++e) r.v[e] = to_e<E>(0.f);
  }
}
template <int V, class E>
__device__ __forceinline__ void rec_st(E* p, int n, const float (&f)[V]) {
  if (V == 2 && n >= 2) {
    if constexpr (V == 2 && sizeof(E) == 2)
      __builtin_nontemporal_store(bf16x2{(bf16)f[0], (bf16)f[1]}, reinterpret_cast<bf16x2_any*>(p));
    else if constexpr (V == 2)
      __builtin_nontemporal_store(f32x2{f[0], f[1]}, reinterpret_cast<f32x2_any*>(p));
  } else {
    p[0] = to_e<E>(f[0]);
  }
}

// Blocks are numbered channels first over the chunks: neighbours read neighbouring lines.
template <int V> __host__ __device__ __forceinline__ uint32_t rec_width(int D) { return ((uint32_t)D + 64 * V - 1) / (64 * V); }
template <int V> __device__ __forceinline__ int rec_chunk(const RecParams& p) { return (int)(blockIdx.x / rec_width<V>(p.D)); }
// Channels of this block: a wave's 64 threads, V each.  false: none for this thread.
template <int V>
__device__ __forceinline__ bool rec_channels(const RecParams& p, int& c, int& n) {
  c = (int)(blockIdx.x % rec_width<V>(p.D) * 64 + (threadIdx.x & 63)) * V;
  n = p.D - c;
  return n > 0;
}
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

constexpr int REC_AHEAD = 8;  // tokens requested together

// The tokens [t0, t1) of one chunk, in order: begin(n) where a sequence starts,
// each(t, x, g, i), finish(n) behind a sequence's last token.  The chunk's rows behind
// the last sequence are not visited.
template <class E, class GT, int V, bool IN, class FB, class FE, class FF>
__device__ __forceinline__ void rec_walk(const RecParams& p, int c, int n, FB begin, FE each, FF finish) {
  const int t0 = rec_chunk<V>(p) * p.chunk, t1 = min(t0 + p.chunk, p.tokens);
  RecSeq s(p);
  if (t0 >= t1 || !s.seek(t0)) return;
  const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c;
  const GT* gp = static_cast<const GT*>(p.g) + t0 * p.g_stride + c;
  const E* ip = static_cast<const E*>(p.i) + (IN ? t0 * p.i_stride + c : 0);
  if (t0 == s.start) begin(s.n);
  for (int t = t0; t < t1; t += REC_AHEAD) {
    RecRaw<E, V> x[REC_AHEAD], i[REC_AHEAD];
    RecRaw<GT, V> g[REC_AHEAD];
#pragma unroll
    for (int k = 0; k < REC_AHEAD; ++k) {
      if (t + k < t1) {
        rec_ld<V>(xp, n, x[k]);
        rec_ld<V>(gp, n, g[k]);
        if (IN) rec_ld<V>(ip, n, i[k]);
      }
      xp += p.x_stride;
      gp += p.g_stride;
      if (IN) ip += p.i_stride;
    }
#pragma unroll
    for (int k = 0; k < REC_AHEAD; ++k) {
      if (t + k >= t1) break;
      if (t + k == s.end) {
        if (!s.next()) return;
        begin(s.n);
      }
      each(t + k, x[k], g[k], i[k]);
      if (t + k == s.end - 1) finish(s.n);
    }
  }
}

// Each chunk's (A, U).
template <class E, class GT, bool SC, bool IN>
__global__ __launch_bounds__(64) void rec_sum_kernel(RecParams p) {
  constexpr int V = kRV<E>;
  int c, n;
  if (!rec_channels<V>(p, c, n)) return;
  float scale[V], A[V], U[V] = {};
  rec_vec<V>(p.scale, 0, p.D, c, n, scale);
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f;
  bool cut = false;
  rec_walk<E, GT, V, IN>(p, c, n,
    [&](int q) {
      cut = true;
      rec_vec<V>(p.h0, q, p.D, c, n, U);
    },
    [&](int, const RecRaw<E, V>& x, const RecRaw<GT, V>& g, const RecRaw<E, V>& i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const RecGate<SC, IN> w(to_f(x.v[e]), to_f(g.v[e]), IN ? to_f(i.v[e]) : 0.f, scale[e]);
        U[e] = fmaf(w.a, U[e], w.u);
        A[e] *= w.a;
      }
    },
    [](int) {});
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < n) p.sum[(int64_t)rec_chunk<V>(p) * p.D + c + e] = make_float2(cut ? -1.f : A[e], U[e]);
}

// The same for the gradient's chain, backwards: carry leaving the chunk's front.
template <class E, class GT, bool SC>
__global__ __launch_bounds__(64) void rec_rev_sum_kernel(RecParams p) {
  constexpr int V = kRV<E>;
  int c, n;
  if (!rec_channels<V>(p, c, n)) return;
  float scale[V], A[V], U[V] = {};
  rec_vec<V>(p.scale, 0, p.D, c, n, scale);
#pragma unroll
  for (int e = 0; e < V; ++e) A[e] = 1.f;
  bool cut = false;  // behind the first sequence's end nothing more reaches the front
  RecParams w = p;   // walks dy in x's place
  w.x = p.dy;
  w.x_stride = p.D;
  rec_walk<E, GT, V, false>(w, c, n, [](int) {},
    [&](int, const RecRaw<E, V>& dy, const RecRaw<GT, V>& g, const RecRaw<E, V>&) {
      if (cut) return;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float L = to_f(g.v[e]);
        if (SC) L = -scale[e] * fast_sigmoid<float>(L);
        A[e] *= __builtin_amdgcn_exp2f(1.44269504f * L);
        U[e] = fmaf(A[e], to_f(dy.v[e]), U[e]);
      }
    },
    [&](int q) {
      if (cut) return;
      cut = true;
      if (!p.dhT) return;
      float d[V];
      rec_vec<V>(p.dhT, q, p.D, c, n, d);
#pragma unroll
      for (int e = 0; e < V; ++e) U[e] = fmaf(A[e], d[e], U[e]);
    });
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < n) p.sum[(int64_t)rec_chunk<V>(p) * p.D + c + e] = make_float2(cut ? -1.f : A[e], U[e]);
}

// States entering the chunks (REV: gradients leaving them): JOIN_S threads a channel
// compose a run of chunks each, then walk it again from what the runs before make.
constexpr int RJ_C = 32, RJ_S = 32;
__device__ __forceinline__ float rec_apply(float2 s, float h) { return s.x < 0.f ? s.y : fmaf(s.x, h, s.y); }
template <bool REV>
__global__ __launch_bounds__(RJ_C * RJ_S) void rec_join_kernel(RecParams p) {
  __shared__ float2 runs[RJ_S][RJ_C + 1];
  const int cl = threadIdx.x % RJ_C, s = threadIdx.x / RJ_C;
  const int c = blockIdx.x * RJ_C + cl;
  const int per = (p.nchunk + RJ_S - 1) / RJ_S, b0 = min(p.nchunk, s * per), b1 = min(p.nchunk, b0 + per);
  auto at = [&](int b) { return (int64_t)(REV ? p.nchunk - 1 - b : b) * p.D + c; };
  float2 r = make_float2(1.f, 0.f);
  if (c < p.D) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
      const float2 v = p.sum[at(b)];
      r = v.x < 0.f ? v : make_float2(r.x < 0.f ? -1.f : r.x * v.x, fmaf(v.x, r.y, v.y));
    }
  }
  runs[s][cl] = r;
  __syncthreads();
  float h = 0.f;
  for (int q = 0; q < s; ++q) h = rec_apply(runs[q][cl], h);
  if (c >= p.D) return;
  float* out = REV ? p.carry : p.enter;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    out[at(b)] = h;
    h = rec_apply(p.sum[at(b)], h);
  }
}

// Blocks past the chunks write the final states of sequences without tokens.
template <int V>
__device__ __forceinline__ bool rec_empty_seq(const RecParams& p, const float* src, float* dst, int c, int n) {
  if (rec_chunk<V>(p) < p.nchunk) return false;
  RecSeq s(p);
  s.n = rec_chunk<V>(p) - p.nchunk;
  s.bounds();
  if (s.end > s.start || !dst) return true;
  float h[V];
  rec_vec<V>(src, s.n, p.D, c, n, h);
  rec_put<V>(dst, s.n, p.D, c, n, h);
  return true;
}

template <class E, class GT, bool SC, bool IN>
__global__ __launch_bounds__(64) void rec_fwd_kernel(RecParams p) {
  constexpr int V = kRV<E>;
  int c, n;
  if (!rec_channels<V>(p, c, n)) return;
  if (rec_empty_seq<V>(p, p.h0, p.hT, c, n)) return;
  float scale[V], h[V];
  rec_vec<V>(p.scale, 0, p.D, c, n, scale);
  rec_vec<V>(p.enter, rec_chunk<V>(p), p.D, c, n, h);
  E* yp = static_cast<E*>(p.y) + c;
  rec_walk<E, GT, V, IN>(p, c, n,
    [&](int q) { rec_vec<V>(p.h0, q, p.D, c, n, h); },
    [&](int t, const RecRaw<E, V>& x, const RecRaw<GT, V>& g, const RecRaw<E, V>& i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const RecGate<SC, IN> w(to_f(x.v[e]), to_f(g.v[e]), IN ? to_f(i.v[e]) : 0.f, scale[e]);
        h[e] = fmaf(w.a, h[e], w.u);
      }
      rec_st<V>(yp + (int64_t)t * p.D, n, h);
    },
    [&](int q) {
      if (p.hT) rec_put<V>(p.hT, q, p.D, c, n, h);
    });
}

// Gradient.  A chunk is one workgroup, a wave to every REC_SUB tokens, whose inputs lie
// in registers: a first walk forms the waves' pairs of both chains, exchanged through
// LDS; a second the states before every token from the state entering; the third goes
// back with the gradient.
template <class E, class GT, bool SC, bool IN>
__global__ __launch_bounds__(512) void rec_bwd_kernel(RecParams p) {
  constexpr int V = kRV<E>, S = REC_SUB;
  __shared__ float2 fw[8][64 * V], bw[8][64 * V];
  int c, n;
  const bool any = rec_channels<V>(p, c, n);
  const int ch = rec_chunk<V>(p);
  if (ch >= p.nchunk) {
    if (any && threadIdx.x < 64) rec_empty_seq<V>(p, p.dhT, p.dh0, c, n);
    return;
  }
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), W = blockDim.x / 64;
  const int t0 = ch * p.chunk + w * S;
  RecSeq s(p);
  const int t1 = min(t0 + S, s.all());
  const bool live = any && t0 < t1 && s.seek(t0);
  const int n0 = s.n;
  RecRaw<E, V> x[S], i[S], dy[S];
  RecRaw<GT, V> g[S];
  float a[S][V], h[S][V], scale[V];
  float2 f[V], b[V];
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = b[e] = make_float2(1.f, 0.f);
  if (live) {
    rec_vec<V>(p.scale, 0, p.D, c, n, scale);
    const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c;
    const GT* gp = static_cast<const GT*>(p.g) + t0 * p.g_stride + c;
    const E* ip = static_cast<const E*>(p.i) + (IN ? t0 * p.i_stride + c : 0);
    const E* dp = static_cast<const E*>(p.dy) + (int64_t)t0 * p.D + c;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (t0 + k < t1) {
        rec_ld<V>(gp + k * p.g_stride, n, g[k]);
        rec_ld<V>(xp + k * p.x_stride, n, x[k]);
        if (IN) rec_ld<V>(ip + k * p.i_stride, n, i[k]);
        rec_ld<V>(dp + (int64_t)k * p.D, n, dy[k]);
      }
    }
    bool cutf = false, cutb = false;
    if (t0 == s.start) {
      cutf = true;
      float t[V];
      rec_vec<V>(p.h0, s.n, p.D, c, n, t);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e].y = t[e];
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (t0 + k >= t1) break;
      if (t0 + k == s.end) {
        if (!s.next()) break;
        cutf = true;
        float t[V];
        rec_vec<V>(p.h0, s.n, p.D, c, n, t);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e].y = t[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const RecGate<SC, IN> q(to_f(x[k].v[e]), to_f(g[k].v[e]), IN ? to_f(i[k].v[e]) : 0.f, scale[e]);
        a[k][e] = q.a;
        h[k][e] = q.u;
        f[e] = make_float2(f[e].x * q.a, fmaf(q.a, f[e].y, q.u));
        if (!cutb) b[e] = make_float2(b[e].x * q.a, fmaf(b[e].x * q.a, to_f(dy[k].v[e]), b[e].y));
      }
      if (t0 + k == s.end - 1 && !cutb) {
        cutb = true;
        float t[V];
        rec_vec<V>(p.dhT, s.n, p.D, c, n, t);
#pragma unroll
        for (int e = 0; e < V; ++e) b[e].y = fmaf(b[e].x, t[e], b[e].y);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (cutf) f[e].x = -1.f;
      if (cutb) b[e].x = -1.f;
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    fw[w][lane * V + e] = f[e];
    bw[w][lane * V + e] = b[e];
  }
  __syncthreads();
  float ds[V] = {};
  if (live) {
    float hc[V], dc[V];
    rec_vec<V>(p.enter, ch, p.D, c, n, hc);
    rec_vec<V>(p.carry, ch, p.D, c, n, dc);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      for (int q = 0; q < w; ++q) hc[e] = rec_apply(fw[q][lane * V + e], hc[e]);
      for (int q = W - 1; q > w; --q) dc[e] = rec_apply(bw[q][lane * V + e], dc[e]);
    }
    // the states before every token
    s.n = n0;
    s.bounds();
    if (t0 == s.start) rec_vec<V>(p.h0, s.n, p.D, c, n, hc);
    int last = t0;  // past the last token that belongs to a sequence
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (t0 + k >= t1) break;
      if (t0 + k == s.end) {
        if (!s.next()) break;
        rec_vec<V>(p.h0, s.n, p.D, c, n, hc);
      }
      last = t0 + k + 1;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = fmaf(a[k][e], hc[e], h[k][e]);
        h[k][e] = hc[e];
        hc[e] = t;
      }
    }
    // back in time
    if (s.n >= s.N || !(last > s.start && last <= s.end)) s.seek(last - 1);
#pragma unroll
    for (int k = S - 1; k >= 0; --k) {
      const int t = t0 + k;
      if (t >= last) continue;
      if (t < s.start) s.seek(t);
      if (t == s.end - 1) rec_vec<V>(p.dhT, s.n, p.D, c, n, dc);
      float dx[V], dg[V], di[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xv = to_f(x[k].v[e]);
        const RecGate<SC, IN> q(xv, to_f(g[k].v[e]), IN ? to_f(i[k].v[e]) : 0.f, scale[e]);
        const float dh = to_f(dy[k].v[e]) + dc[e], dhs = IN ? dh * q.si : dh;
        dc[e] = a[k][e] * dh;
        dx[e] = SC ? dhs * q.m : dhs;
        di[e] = dx[e] * xv * (1.f - q.si);
        float dl = dc[e] * h[k][e];
        if (SC) {
          dl -= dhs * xv * (q.a * q.a) * q.im;
          dg[e] = -dl * scale[e] * (q.sg - q.sg * q.sg);
          ds[e] -= dl * q.sg;
        } else {
          dg[e] = dl;
        }
      }
      rec_st<V>(static_cast<E*>(p.dx) + (int64_t)t * p.D + c, n, dx);
      rec_st<V>(static_cast<GT*>(p.dg) + (int64_t)t * p.D + c, n, dg);
      if (IN) rec_st<V>(static_cast<E*>(p.di) + (int64_t)t * p.D + c, n, di);
      if (t == s.start && p.dh0) rec_put<V>(p.dh0, s.n, p.D, c, n, dc);
    }
  }
  if (!SC) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e) fw[w][lane * V + e].x = ds[e];
  __syncthreads();
  if (w == 0 && any) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float t = 0.f;
      for (int q = 0; q < W; ++q) t += fw[q][lane * V + e].x;
      ds[e] = t;
    }
    rec_put<V>(p.part, ch, p.D, c, n, ds);
  }
}

template <class E, class GT, bool SC, bool IN>
__global__ __launch_bounds__(64) void rec_step_kernel(RecStepParams p) {
  constexpr int V = kRV<E>;
  const uint32_t wide = rec_width<V>(p.D);
  const int c = (int)(blockIdx.x % wide * 64 + threadIdx.x) * V, n = p.D - c, r = (int)(blockIdx.x / wide);
  if (n <= 0) return;
  const int slot = p.state_idx ? p.state_idx[r] : r;
  if (slot < 0 || slot >= p.num_slots) return;
  RecRaw<E, V> x, i;
  RecRaw<GT, V> g;
  rec_ld<V>(static_cast<const E*>(p.x) + r * p.x_stride + c, n, x);
  rec_ld<V>(static_cast<const GT*>(p.g) + r * p.g_stride + c, n, g);
  if (IN) rec_ld<V>(static_cast<const E*>(p.i) + r * p.i_stride + c, n, i);
  float h[V], scale[V];
  rec_vec<V>(p.state, slot, p.D, c, n, h);
  rec_vec<V>(p.scale, 0, p.D, c, n, scale);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const RecGate<SC, IN> w(to_f(x.v[e]), to_f(g.v[e]), IN ? to_f(i.v[e]) : 0.f, scale[e]);
    h[e] = fmaf(w.a, h[e], w.u);
  }
  rec_put<V>(p.state, slot, p.D, c, n, h);
  rec_st<V>(static_cast<E*>(p.y) + (int64_t)r * p.D + c, n, h);
}

// f<E, GT, SC, IN>() by the call's types and optional inputs.
template <class E, class GT, class F>
void rec_pick(bool sc, bool in, F f) {
  if (sc && in) f.template operator()<E, GT, true, true>();
  else if (sc) f.template operator()<E, GT, true, false>();
  else if (in) f.template operator()<E, GT, false, true>();
  else f.template operator()<E, GT, false, false>();
}
template <class F>
hipError_t rec_types(int dtype, int g_f32, bool sc, bool in, F f) {
  if (dtype == GDN_F32) rec_pick<float, float>(sc, in, f);
  else if (g_f32) rec_pick<bf16, float>(sc, in, f);
  else rec_pick<bf16, bf16>(sc, in, f);
  return hipGetLastError();
}
struct RecLaunch {
  enum { SUM, RSUM, FWD, BWD } what;
  const RecParams& p;
  hipStream_t st;
  template <class E, class GT, bool SC, bool IN>
  void operator()() const {
    const int more = what == FWD && p.hT || what == BWD && p.dh0 ? p.N : 0;
    const dim3 grid(rec_width<kRV<E>>(p.D) * (uint32_t)(p.nchunk + more));
    if (grid.x == 0) return;
    if (what == SUM) hipLaunchKernelGGL((rec_sum_kernel<E, GT, SC, IN>), grid, dim3(64), 0, st, p);
    else if (what == RSUM) hipLaunchKernelGGL((rec_rev_sum_kernel<E, GT, SC>), grid, dim3(64), 0, st, p);
    else if (what == FWD) hipLaunchKernelGGL((rec_fwd_kernel<E, GT, SC, IN>), grid, dim3(64), 0, st, p);
    else hipLaunchKernelGGL((rec_bwd_kernel<E, GT, SC, IN>), grid, dim3(64 * (p.chunk / REC_SUB)), 0, st, p);
  }
};
struct RecStepLaunch {
  const RecStepParams& p;
  hipStream_t st;
  template <class E, class GT, bool SC, bool IN>
  void operator()() const {
    const dim3 grid(rec_width<kRV<E>>(p.D) * (uint32_t)p.N);
    hipLaunchKernelGGL((rec_step_kernel<E, GT, SC, IN>), grid, dim3(64), 0, st, p);
  }
};

}  // namespace

hipError_t launch_rec_sum(int dtype, const RecParams& p, bool rev, hipStream_t st) {
  return rec_types(dtype, p.g_f32, p.scale, p.i, RecLaunch{rev ? RecLaunch::RSUM : RecLaunch::SUM, p, st});
}
hipError_t launch_rec_join(const RecParams& p, bool rev, hipStream_t st) {
  const dim3 grid((p.D + RJ_C - 1) / RJ_C);
  if (rev) hipLaunchKernelGGL((rec_join_kernel<true>), grid, dim3(RJ_C * RJ_S), 0, st, p);
  else hipLaunchKernelGGL((rec_join_kernel<false>), grid, dim3(RJ_C * RJ_S), 0, st, p);
  return hipGetLastError();
}
hipError_t launch_rec_fwd(int dtype, const RecParams& p, hipStream_t st) {
  return rec_types(dtype, p.g_f32, p.scale, p.i, RecLaunch{RecLaunch::FWD, p, st});
}
hipError_t launch_rec_bwd(int dtype, const RecParams& p, hipStream_t st) {
  return rec_types(dtype, p.g_f32, p.scale, p.i, RecLaunch{RecLaunch::BWD, p, st});
}
hipError_t launch_rec_step(int dtype, const RecStepParams& p, hipStream_t st) {
  return rec_types(dtype, p.g_f32, p.scale, p.i, RecStepLaunch{p, st});
}

}  // namespace gdn
