// k_latent_simt.cu -- absorbed and expanded latent attention on the CUDA
// cores: every dtype, width and alignment, and the join of shared items.
//
// One pass over the tokens with a running maximum m and sum l per head:
//   m' = max(m, s_j),  l' = l 2^(m - m') + sum 2^(s_j - m'),
//   o' = o 2^(m - m') + sum 2^(s_j - m') v_j
// in log2 units (the softmax scale carries log2 e), everything in fp32.
// Bound by shared memory, which each multiply-add of a score reads twice: at 96
// requests x 128 heads x 2048 slots 14.5 ms (3.8 TFLOP/s; before queries and
// weights were read four at a time); at what it is for, one
// fp32 request of 8 heads with 256 slots of 320, 13 us, most of that the start
// and the join.
#include "latent_internal.cuh"

namespace spin {
namespace {

constexpr int kThreads = 256;
constexpr int kNH = kSimtHeads, kT = kSimtTile;
constexpr float kNegInf = -INFINITY;

// The running softmax of kNH query vectors over tiles of kT tokens.  Warp h
// owns vector h's statistics; thread i the output columns i and i + 256.
// kv rows in shared memory have an odd stride, so a column read across tokens
// has no bank conflicts.
struct Tile {
  float* q;     // [kNH][W]
  float* kv;    // [kT][stride]
  float* p;     // [kT][kNH]
  float* alpha; // [kNH]
  int W, stride, voff, dv;

  // Scores of this thread's (vector warp, token lane), the running softmax
  // and the output update.  `seen`: whether this vector attends to this token.
  __device__ __forceinline__ void step(float& m, float& l, float (&o)[2][kNH], float scale, bool seen) const {
    const int h = threadIdx.x >> 5, j = threadIdx.x & 31;
    const float* qh = q + h * W;
    const float* kj = kv + j * stride;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 4
    for (int i = 0; i < W; i += 4) {  // W is a multiple of 8
      const float4 x = *reinterpret_cast<const float4*>(qh + i);
      s0 = fmaf(x.x, kj[i], s0);
      s1 = fmaf(x.y, kj[i + 1], s1);
      s2 = fmaf(x.z, kj[i + 2], s2);
      s3 = fmaf(x.w, kj[i + 3], s3);
    }
    const float s = seen ? ((s0 + s1) + (s2 + s3)) * scale : kNegInf;
    float mt = s;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
    const float mn = fmaxf(m, mt);
    const float ref = mn == kNegInf ? 0.f : mn;  // nothing seen yet: every weight 0
    const float e = seen ? exp2f(s - ref) : 0.f;
    const float al = exp2f(m - ref);
    float sum = e;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * al + sum;
    m = mn;
    p[j * kNH + h] = e;
    if (j == 0) alpha[h] = al;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = threadIdx.x + c * kThreads;
      if (d >= dv) continue;
#pragma unroll
      for (int h2 = 0; h2 < kNH; ++h2) o[c][h2] *= alpha[h2];
      const float* v = kv + voff + d;
#pragma unroll 4
      for (int t = 0; t < kT; ++t) {
        const float x = v[t * stride];
        float w[kNH];
#pragma unroll
        for (int k = 0; k < kNH; k += 4)
          *reinterpret_cast<float4*>(w + k) = *reinterpret_cast<const float4*>(p + t * kNH + k);
        // a weight of exactly 0 takes nothing from the token, whatever it holds
#pragma unroll
        for (int h2 = 0; h2 < kNH; ++h2) o[c][h2] = w[h2] != 0.f ? fmaf(w[h2], x, o[c][h2]) : o[c][h2];
      }
    }
    __syncthreads();
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_attn_simt(const __grid_constant__ AttnArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) float sm[];
  const LatentCache& C = a.cache;
  const int W = C.dc + C.dr;
  Tile t{sm, sm + kNH * W, nullptr, nullptr, W, W + 1, 0, C.dc};
  t.p = t.kv + kT * t.stride;
  t.alpha = t.p + kNH * kT;
  int64_t* row = reinterpret_cast<int64_t*>(sm + ((t.alpha + kNH - sm + 1) / 2 * 2));  // [kT] cache rows, -1: none
  __shared__ int tmp[36];
  __shared__ float norm[kNH];
  const int g = blockIdx.x % a.ngroups, u = blockIdx.x / a.ngroups;
  const int h0 = g * kNH, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place at0 = attn_place(a, -1, u, tmp);
  if (u >= at0.ranges) return;
  const int my_begin = range_begin(at0.total, at0.ranges, u), stop = range_begin(at0.total, at0.ranges, u + 1);
  int item = at0.item, first = at0.first, at = my_begin;
  while (at < stop) {
    const int q = item / a.rows, r = item - q * a.rows;
    const int end = attn_end(a, q, r);
    if (end == 0 && threadIdx.x == 0) raise_error(a.err, ERR_CTX_LEN, q, (uint32_t)a.ctx_len[q]);
    const int n = attn_tiles(a, end);
    const int t0 = at - first, t1 = min(n, stop - first);
    __syncthreads();
    {
      const int h = h0 + warp;
      const T* ql = reinterpret_cast<const T*>(a.ql) + item * a.ql_tok + h * a.ql_head;
      const T* qr = reinterpret_cast<const T*>(a.qr) + item * a.qr_tok + h * a.qr_head - C.dc;
#pragma unroll 4
      for (int d = lane; d < W; d += 32) t.q[warp * W + d] = h < a.H ? to_f32(d < C.dc ? ql[d] : qr[d]) : 0.f;
    }
    float m = kNegInf, l = 0.f, o[2][kNH] = {};
    for (int k = t0; k < t1; ++k) {
      if (warp == 0) {
        const int e = k * kT + lane;
        int slot = -1;
        if (a.list) {
          if (e < a.topk) slot = a.list[(int64_t)item * a.topk + e];
        } else {
          slot = e;
        }
        row[lane] = (slot >= 0 && slot < end) ? cache_row(C, q, slot, a.err) : -1;
      }
      __syncthreads();
      // a warp takes tokens warp, warp + 8, ..: all four of one piece in flight at once
      constexpr int V = 16 / (int)sizeof(T);
      const bool vec = ((uintptr_t)C.data & 15) == 0 && W % V == 0;
      for (int d = lane * (vec ? V : 1); d < W; d += 32 * (vec ? V : 1)) {
        uint4 x[kT / 8];
#pragma unroll
        for (int i = 0; i < kT / 8; ++i) {
          const int64_t r = row[warp + 8 * i];
          x[i] = make_uint4(0, 0, 0, 0);
          if (r >= 0) {
            const T* src = reinterpret_cast<const T*>(C.data) + r * W + d;
            if (vec)
              x[i] = *reinterpret_cast<const uint4*>(src);
            else
              *reinterpret_cast<T*>(&x[i]) = *src;
          }
        }
#pragma unroll
        for (int i = 0; i < kT / 8; ++i) {
          const T* e = reinterpret_cast<const T*>(&x[i]);
          float* dst = t.kv + (warp + 8 * i) * t.stride + d;
#pragma unroll
          for (int k = 0; k < V; ++k)
            if (vec || k == 0) dst[k] = to_f32(e[k]);
        }
      }
      const bool seen = row[lane] >= 0;
      __syncthreads();
      t.step(m, l, o, a.scale_log2, seen);
    }
    if (t0 == 0 && t1 == n) {
      if (lane == 0) {
        norm[warp] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        if (a.lse && h0 + warp < a.H)
          a.lse[(int64_t)item * a.H + h0 + warp] = l == 0.f ? kNegInf : (m + log2f(l)) * (1.f / kLog2e);
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = threadIdx.x + c * kThreads;
        if (d < C.dc)
          for (int h = 0; h < kNH && h0 + h < a.H; ++h)
            reinterpret_cast<T*>(a.out)[((int64_t)item * a.H + h0 + h) * C.dc + d] = from_f32<T>(o[c][h] * norm[h]);
      }
    } else {
      const int64_t part = (int64_t)blockIdx.x * 2 + (first <= my_begin ? 0 : 1);
      if (lane == 0) a.part_ml[part * kNH + warp] = make_float2(m, l);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = threadIdx.x + c * kThreads;
        if (d < C.dc)
#pragma unroll
          for (int h = 0; h < kNH; ++h) a.part[(part * kNH + h) * C.dc + d] = o[c][h];
      }
    }
    at = first + t1;
    first += n;
    ++item;
  }
}

// Joins the shares of an item that several blocks worked on, WPH warps per
// (item, head) of kJoinWarps: warp i of a head takes shares i, i + WPH, ..,
// and the warps' sums meet in warp order.  Bound by the shares' bytes (10 MB for 8
// contexts x 32 heads: 8.8 us alone from a cold L2), or for one long context by
// the latency of its many shares (hence WPH = 8 there).
constexpr int kJoinWarps = 8;

template <typename T, int WPH>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_combine(const __grid_constant__ AttnArgs a) {
  __shared__ int tmp[36];
  __shared__ float4 sums[WPH > 1 ? kJoinWarps : 1][WPH > 1 ? 128 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = a.whole * a.ranges + blockIdx.y, h = blockIdx.x * (kJoinWarps / WPH) + warp / WPH, mine = warp % WPH;
  // The lengths were there before the attention kernel started, so the place
  // of the shares is found while it still runs.
  const Place at = attn_place(a, item, 0, tmp);
  const int total = at.total, ranges = at.ranges, first = at.first;
  const int n = attn_tiles(a, attn_end(a, item / a.rows, item % a.rows));
  const int u0 = range_of(total, ranges, first), u1 = range_of(total, ranges, first + n - 1);
  pdl_enter();
  if (u0 == u1 || h >= a.H) return;  // (WPH = 8: the same for all warps of the block)
  const int g = h / a.group, hh = h - g * a.group, dc = a.cache.dc;
  // the item starts inside its first block's range, or with it; it ran on into the others'
  const int head = first == range_begin(total, ranges, u0) ? 0 : 1;
  auto slot = [&](int u) {
    return ((int64_t)(u * a.ngroups + g) * 2 + (u == u0 ? head : 0)) * a.group + hh;
  };
  // columns 4 (lane + 32 i) .. + 3 of kAhead shares at a time; the first ones' loads go out before the weights are
  // known
  constexpr int kAhead = 4;
  float4 x[4][kAhead];
  auto fetch = [&](int v) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const float4* src = reinterpret_cast<const float4*>(a.part + slot(min(v + k * WPH, u1)) * dc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * (lane + 32 * i) < dc) x[i][k] = src[lane + 32 * i];
    }
  };
  fetch(u0 + mine);
  float m = kNegInf;
  for (int u = u0 + lane; u <= u1; u += 32) m = fmaxf(m, a.part_ml[slot(u)].x);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float ref = m == kNegInf ? 0.f : m;
  float l = 0.f;
  for (int u = u0 + lane; u <= u1; u += 32) {
    const float2 ml = a.part_ml[slot(u)];
    l += ml.y * exp2f(ml.x - ref);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float norm = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (mine == 0 && lane == 0 && a.lse)
    a.lse[(int64_t)item * a.H + h] = l == 0.f ? kNegInf : (m + log2f(l)) * (1.f / kLog2e);
  float4 o[4] = {};
  for (int v = u0 + mine; v <= u1; v += WPH * kAhead) {
    if (v != u0 + mine) fetch(v);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = v + k * WPH;
      const float w = u <= u1 ? exp2f(a.part_ml[slot(u)].x - ref) : 0.f;
      if (w == 0.f) continue;  // (a share without weight may hold anything)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i].x = fmaf(w, x[i][k].x, o[i].x);
        o[i].y = fmaf(w, x[i][k].y, o[i].y);
        o[i].z = fmaf(w, x[i][k].z, o[i].z);
        o[i].w = fmaf(w, x[i][k].w, o[i].w);
      }
    }
  }
  const bool aligned = ((uintptr_t)a.out & 15) == 0;
  auto store = [&](int c, float4 x) {
    struct alignas(4 * sizeof(T)) Four {
      T v[4];
    } f{{from_f32<T>(x.x * norm), from_f32<T>(x.y * norm), from_f32<T>(x.z * norm), from_f32<T>(x.w * norm)}};
    T* out = reinterpret_cast<T*>(a.out) + ((int64_t)item * a.H + h) * dc + 4 * c;
    if (aligned) {
      *reinterpret_cast<Four*>(out) = f;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) out[k] = f.v[k];
    }
  };
  if constexpr (WPH == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * (lane + 32 * i) < dc) store(lane + 32 * i, o[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][lane + 32 * i] = o[i];
    __syncthreads();
    for (int c = threadIdx.x; 4 * c < dc; c += kJoinWarps * 32) {
      float4 x = sums[0][c];
      for (int k = 1; k < kJoinWarps; ++k) {
        const float4 y = sums[k][c];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      store(c, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Expanded form
// ---------------------------------------------------------------------------
constexpr int kES = 32, kEK = 32;  // slots of a block, reduction step
constexpr int kEStride = kES + 4;  // of a step's slots in shared memory: 16-byte aligned, spread over banks

// kv[h][off + s] = W_h c_s for a tile of kES slots and one head; head 0 also
// copies the shared key part.  grid (slot tiles, heads, requests).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_expand_simt(const __grid_constant__ PrefillArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) float sm[];
  __shared__ int64_t tmp[33];
  __shared__ int64_t row[kES];
  const LatentCache& C = a.cache;
  const int h = blockIdx.y, q = blockIdx.z, N = a.dn + a.dv, W = C.dc + C.dr;
  const Chunk ch = prefill_chunk(a, q, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (ch.end == 0) return;
  const int64_t off = prefill_rows_before(a, q, tmp);
  if (off + ch.end > a.cap) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) raise_error(a.err, ERR_CAPACITY, q, (uint32_t)ch.end);
    return;
  }
  float* cs = sm;                    // [kEK][kEStride]
  float* ws = sm + kEK * kEStride;  // [N][kEK + 1]
  for (int s0 = blockIdx.x * kES; s0 < ch.end; s0 += gridDim.x * kES) {
    __syncthreads();
    if (threadIdx.x < kES) {
      const int slot = s0 + threadIdx.x;
      row[threadIdx.x] = slot < ch.end ? cache_row(C, q, slot, a.err) : -1;
    }
    __syncthreads();
    float acc[2][kES] = {};
    for (int k0 = 0; k0 < C.dc; k0 += kEK) {
      for (int i = threadIdx.x; i < kES * kEK; i += kThreads) {
        const int s = i / kEK, k = i % kEK;
        cs[k * kEStride + s] = (row[s] >= 0 && k0 + k < C.dc)
                                    ? to_f32(reinterpret_cast<const T*>(C.data)[row[s] * W + k0 + k]) : 0.f;
      }
      for (int i = threadIdx.x; i < N * kEK; i += kThreads) {
        const int n = i / kEK, k = i % kEK;
        ws[n * (kEK + 1) + k] = k0 + k < C.dc
            ? to_f32(reinterpret_cast<const T*>(a.w)[((int64_t)h * N + n) * C.dc + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = threadIdx.x + c * kThreads;
        if (n < N)
          for (int k = 0; k < kEK; ++k) {
            const float w = ws[n * (kEK + 1) + k];
#pragma unroll
            for (int s = 0; s < kES; s += 4) {
              const float4 x = *reinterpret_cast<const float4*>(cs + k * kEStride + s);
              acc[c][s] = fmaf(w, x.x, acc[c][s]);
              acc[c][s + 1] = fmaf(w, x.y, acc[c][s + 1]);
              acc[c][s + 2] = fmaf(w, x.z, acc[c][s + 2]);
              acc[c][s + 3] = fmaf(w, x.w, acc[c][s + 3]);
            }
          }
      }
      __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = threadIdx.x + c * kThreads;
      if (n < N)
#pragma unroll
        for (int s = 0; s < kES; ++s)
          if (s0 + s < ch.end)
            reinterpret_cast<T*>(a.kv)[(h * a.cap + off + s0 + s) * N + n] = from_f32<T>(acc[c][s]);
    }
    if (h == 0)
      for (int i = threadIdx.x; i < kES * C.dr; i += kThreads) {
        const int s = i / C.dr, d = i - s * C.dr;
        if (row[s] >= 0)
          reinterpret_cast<T*>(a.kr)[(off + s0 + s) * C.dr + d] =
              reinterpret_cast<const T*>(C.data)[row[s] * W + C.dc + d];
      }
  }
}

// Whether a page of the request's first `end` slots lies outside the cache
// (all threads of the block).
__device__ __forceinline__ bool bad_pages(const LatentCache& C, int q, int end) {
  int bad = 0;
  for (int i = threadIdx.x; i <= (end - 1) >> C.log2b; i += blockDim.x) {
    const int page = C.bt[(int64_t)q * C.bt_stride + i];
    bad |= page < 0 || page >= C.num_pages;
  }
  return __syncthreads_or(bad) != 0;
}

// Causal attention of kNH rows of one head.  grid (row tiles, heads, requests).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_prefill_simt(const __grid_constant__ PrefillArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) float sm[];
  __shared__ int64_t tmp[33];
  __shared__ float norm[kNH];
  const int h = blockIdx.y, q = blockIdx.z, N = a.dn + a.dv, dr = a.cache.dr, W = a.dn + dr;
  const Chunk ch = prefill_chunk(a, q, false);
  if (ch.end == 0) return;
  const int64_t off = prefill_rows_before(a, q, tmp);
  if (off + ch.end > a.cap || bad_pages(a.cache, q, ch.end)) return;
  Tile t{sm, sm + kNH * W, nullptr, nullptr, W, (W + a.dv) | 1, W, a.dv};
  t.p = t.kv + kT * t.stride;
  t.alpha = t.p + kNH * kT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token0 = (int64_t)q * a.rows;
  for (int r0 = blockIdx.x * kNH; r0 < ch.count; r0 += gridDim.x * kNH) {
    __syncthreads();
    {
      const T* x = reinterpret_cast<const T*>(a.q) + (token0 + r0 + warp) * a.q_tok + h * a.q_head;
#pragma unroll 4
      for (int d = lane; d < W; d += 32) t.q[warp * W + d] = r0 + warp < ch.count ? to_f32(x[d]) : 0.f;
    }
    const int pos = ch.ctx - 1 + r0 + warp;
    const int last = min(ch.ctx - 1 + r0 + kNH - 1, ch.end - 1);
    float m = kNegInf, l = 0.f, o[2][kNH] = {};
    for (int j0 = 0; j0 <= last; j0 += kT) {
      __syncthreads();
      // 16 bytes a lane (all widths are multiples of 8), a warp's four slots at once
      constexpr int V = 16 / (int)sizeof(T);
      const T* kv = reinterpret_cast<const T*>(a.kv) + (h * a.cap + off + j0 + warp) * N;
      const T* kr = reinterpret_cast<const T*>(a.kr) + (off + j0 + warp) * dr;
      for (int d = lane * V; d < W + a.dv; d += 32 * V) {
        const T* src = d < a.dn ? kv + d : d < W ? kr + (d - a.dn) : kv + (d - dr);
        const int64_t step = 8 * (d < a.dn || d >= W ? N : dr);
        uint4 x[kT / 8];
#pragma unroll
        for (int i = 0; i < kT / 8; ++i)
          x[i] = j0 + warp + 8 * i < ch.end ? *reinterpret_cast<const uint4*>(src + i * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kT / 8; ++i) {
          const T* e = reinterpret_cast<const T*>(&x[i]);
          float* dst = t.kv + (warp + 8 * i) * t.stride + d;
#pragma unroll
          for (int k = 0; k < V; ++k) dst[k] = to_f32(e[k]);
        }
      }
      __syncthreads();
      t.step(m, l, o, a.scale_log2, j0 + lane <= pos && j0 + lane <= last);
    }
    if (lane == 0) norm[warp] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = threadIdx.x + c * kThreads;
      if (d < a.dv)
        for (int r = 0; r < kNH && r0 + r < ch.count; ++r)
          reinterpret_cast<T*>(a.out)[((token0 + r0 + r) * a.H + h) * a.dv + d] = from_f32<T>(o[c][r] * norm[r]);
    }
  }
}

// Shared memory of a block; the largest dims take less than kMaxSmem.
constexpr int kMaxSmem = 160 * 1024;
size_t attn_smem(int W) {
  return sizeof(float) * (kNH * W + kT * (W + 1) + kNH * kT + kNH + 2) + sizeof(int64_t) * kT;
}
size_t expand_smem(int N) { return sizeof(float) * (kEK * kEStride + (size_t)N * (kEK + 1)); }
size_t prefill_smem(int W, int dv) { return sizeof(float) * (kNH * W + kT * ((W + dv) | 1) + kNH * kT + kNH); }

template <typename T>
cudaError_t raise_limits() {
  cudaError_t e = cudaFuncSetAttribute(k_attn_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_expand_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_prefill_simt<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  return e;
}

}  // namespace

cudaError_t prepare_attn_simt() {
  const cudaError_t e = raise_limits<float>();
  return e == cudaSuccess ? raise_limits<__nv_bfloat16>() : e;
}

cudaError_t launch_attn_simt(const AttnArgs& a, int bf16, cudaStream_t s) {
  const int W = a.cache.dc + a.cache.dr;
  const size_t smem = attn_smem(W);
  auto kernel = bf16 ? k_attn_simt<__nv_bfloat16> : k_attn_simt<float>;
  PdlLaunch l(dim3((unsigned)(a.ranges * a.ngroups)), dim3(kThreads), smem, s);
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

cudaError_t launch_attn_combine(const AttnArgs& a, int bf16, cudaStream_t s) {
  // By an item's shares, at the even lengths of lists.  One warp a head or eight, the whole call: 9 shares each (16
  // contexts of 4096, 16 heads) 30.7 and 28.5 us, 18 (8 contexts up to 32K, 32 heads) 61.6 and 50.4 us, 6 (24
  // contexts of 4096, 32 heads) 43.9 and 50.6 us.
  const int items = a.Q * a.rows - a.whole * a.ranges;
  const bool many = a.rest > 8 * items;
  const int per = many ? 1 : kJoinWarps;
  auto kernel = many ? (bf16 ? k_attn_combine<__nv_bfloat16, kJoinWarps> : k_attn_combine<float, kJoinWarps>)
                     : (bf16 ? k_attn_combine<__nv_bfloat16, 1> : k_attn_combine<float, 1>);
  PdlLaunch l(dim3((unsigned)((a.H + per - 1) / per), (unsigned)items), dim3(kJoinWarps * 32), 0, s);
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

cudaError_t launch_expand_simt(const PrefillArgs& a, int bf16, cudaStream_t s) {
  const size_t smem = expand_smem(a.dn + a.dv);
  auto kernel = bf16 ? k_expand_simt<__nv_bfloat16> : k_expand_simt<float>;
  const int64_t tiles = ((int64_t)a.max_slots + kES - 1) / kES;
  PdlLaunch l(dim3((unsigned)(tiles < 1024 ? tiles : 1024), (unsigned)a.H, (unsigned)a.Q), dim3(kThreads), smem, s);
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

cudaError_t launch_prefill_simt(const PrefillArgs& a, int bf16, cudaStream_t s) {
  const int W = a.dn + a.cache.dr;
  const size_t smem = prefill_smem(W, a.dv);
  auto kernel = bf16 ? k_prefill_simt<__nv_bfloat16> : k_prefill_simt<float>;
  const int64_t tiles = ((int64_t)a.rows + kNH - 1) / kNH;
  PdlLaunch l(dim3((unsigned)(tiles < 4096 ? tiles : 4096), (unsigned)a.H, (unsigned)a.Q), dim3(kThreads), smem, s);
  // Not scheduled beside the expansion: its blocks would gather on the SMs that have room early (126 us, not 87, for 3
  // x 150 fp32 rows on 400 slots x 5 heads).
  l.cfg.numAttrs = 0;
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

}  // namespace spin
