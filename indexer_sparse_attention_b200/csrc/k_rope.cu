// k_rope.cu -- rotary positions, and the append of new tokens to the paged
// latent cache.
//
// A pair (x, y) of a head turns by the angle t of its position:
//   (x cos t - y sin t, x sin t + y cos t),
// computed in fp32 from the stored values and rounded once.  Both kernels
// move each byte once and compute little: they are bound by HBM, and at
// decode sizes by the latency of one dependent load (position), the sine and
// the store.
#include <algorithm>

#include "latent_internal.cuh"

namespace spin {
namespace {

constexpr int kRopeThreads = 128;

// (products and sums spelled out, so that every kernel gives the same bits)
template <typename T>
__device__ __forceinline__ void turn_pair(T& x, T& y, float2 cs) {
  const float a = to_f32(x), b = to_f32(y);
  x = from_f32<T>(__fmaf_rn(a, cs.x, -__fmul_rn(b, cs.y)));
  y = from_f32<T>(__fmaf_rn(a, cs.y, __fmul_rn(b, cs.x)));
}

// 16 bytes of elements.
template <typename T>
struct alignas(16) Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
  T v[kN];
};

// 16-byte pieces.  A block takes one token and a range of its heads: first the
// pieces that are only copied, which need no sines, then the rotated ones (a
// vector, or in the half layout two half a rotation apart).  One piece a
// thread and step at full occupancy: 34 us for 8192 tokens x 32 heads x 192 in
// the half layout (5.9 TB/s); four pieces a thread at 116 registers took 108 us,
// blocks of 256 threads 36 us, rotating and copying in one loop 43 us.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 16) k_rope_vec(const __grid_constant__ RopeArgs a, int heads_per_block) {
  constexpr int V = Vec<T>::kN;
  pdl_enter();
  __shared__ float2 cs[kMaxRopeDim / 2];
  const int64_t t = blockIdx.x;
  const int h0 = blockIdx.y * heads_per_block, heads = min(heads_per_block, a.heads - h0);
  const int d2 = a.rope_dim / 2, turned = HALF ? d2 / V : a.rope_dim / V;
  const T* x = reinterpret_cast<const T*>(a.x) + t * a.x_tok + h0 * a.x_head;
  T* o = reinterpret_cast<T*>(a.out) + t * a.o_tok + h0 * a.o_head;
  if ((int)threadIdx.x < d2) cs[threadIdx.x] = rope_cos_sin(a.tab.turn[threadIdx.x], a.pos[t], a.tab.mul);
  if (a.out != a.x) {
    const int copied = (a.head_dim - a.rope_dim) / V;
#pragma unroll 2
    for (int u = threadIdx.x; u < heads * copied; u += kRopeThreads) {
      const int h = u / copied;
      int e = (u - h * copied) * V;
      if (e >= a.offset) e += a.rope_dim;
      *reinterpret_cast<Vec<T>*>(o + h * a.o_head + e) = *reinterpret_cast<const Vec<T>*>(x + h * a.x_head + e);
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < heads * turned; u += kRopeThreads) {
    const int h = u / turned, i = u - h * turned, e0 = a.offset + i * V;
    const T* src = x + h * a.x_head + e0;
    T* dst = o + h * a.o_head + e0;
    Vec<T> p = *reinterpret_cast<const Vec<T>*>(src);
    if (HALF) {
      Vec<T> q = *reinterpret_cast<const Vec<T>*>(src + d2);
#pragma unroll
      for (int e = 0; e < V; ++e) turn_pair(p.v[e], q.v[e], cs[i * V + e]);
      *reinterpret_cast<Vec<T>*>(dst + d2) = q;
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) turn_pair(p.v[e], p.v[e + 1], cs[(i * V + e) / 2]);
    }
    *reinterpret_cast<Vec<T>*>(dst) = p;
  }
}

// One element pair or one copied element per thread and step: any strides,
// alignment and dims (131 us where the kernel above takes 34).
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) k_rope_any(const __grid_constant__ RopeArgs a) {
  pdl_enter();
  const int d2 = a.rope_dim / 2;
  const bool in_place = a.out == a.x;
  const int plain = in_place ? 0 : a.head_dim - a.rope_dim;
  const int per_head = d2 + plain;
  __shared__ float2 cs[kMaxRopeDim / 2];
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    __syncthreads();
    if ((int)threadIdx.x < d2) cs[threadIdx.x] = rope_cos_sin(a.tab.turn[threadIdx.x], a.pos[t], a.tab.mul);
    __syncthreads();
    const T* x = reinterpret_cast<const T*>(a.x) + t * a.x_tok;
    T* o = reinterpret_cast<T*>(a.out) + t * a.o_tok;
    for (int u = blockIdx.y * kRopeThreads + threadIdx.x; u < a.heads * per_head; u += gridDim.y * kRopeThreads) {
      const int h = u / per_head, i = u - h * per_head;
      const T* xh = x + h * a.x_head;
      T* oh = o + h * a.o_head;
      if (i < d2) {
        const int e0 = a.offset + (a.half ? i : 2 * i), e1 = a.offset + (a.half ? i + d2 : 2 * i + 1);
        T v0 = xh[e0], v1 = xh[e1];
        turn_pair(v0, v1, cs[i]);
        oh[e0] = v0;
        oh[e1] = v1;
      } else {
        const int e = i - d2 < a.offset ? i - d2 : i - d2 + a.rope_dim;
        oh[e] = xh[e];
      }
    }
  }
}

// New tokens into the cache, 16-byte pieces: one warp per token.  96 requests'
// tokens 2.0 us, 8 ragged chunks of up to 1024 4.1 us (element by element, as
// below, 4.8 and 8.4 us): latency of length, page and store.
template <typename T, bool HALF>
__global__ void __launch_bounds__(256) k_append_vec(const __grid_constant__ AppendArgs a) {
  constexpr int V = Vec<T>::kN;
  constexpr int kC = 512 / V / 32;  // pieces of the latent a lane takes at most
  pdl_enter();
  __shared__ float2 cs_all[8][kMaxRopeDim / 2];
  const int lane = threadIdx.x & 31;
  float2* cs = cs_all[threadIdx.x >> 5];
  const LatentCache& C = a.cache;
  const int d2 = C.dr / 2, turned = HALF ? d2 / V : C.dr / V;
  const int64_t n = (int64_t)a.Q * a.rows;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * 8) {
    const int q = (int)(t / a.rows), r = (int)(t - (int64_t)q * a.rows);
    const int ctx = a.ctx_len[q];
    const int count = a.row_count ? a.row_count[q] : a.rows;
    if (count < 0 || count > a.rows) {
      if (r == 0 && lane == 0) raise_error(a.err, ERR_ACCEPTED, q, (uint32_t)count);
      continue;
    }
    if (count == 0) continue;  // (an idle request's ctx_len is not looked at)
    if (ctx < 1 || (int64_t)ctx - 1 + count > a.max_slots) {
      if (r == 0 && lane == 0) raise_error(a.err, ERR_CTX_LEN, q, (uint32_t)ctx);
      continue;
    }
    if (r >= count) continue;
    const int slot = ctx - 1 + r;
    const int page = C.bt[(int64_t)q * C.bt_stride + (slot >> C.log2b)];
    // the token's pieces, while the page's number is on its way
    const Vec<T>* c = reinterpret_cast<const Vec<T>*>(reinterpret_cast<const T*>(a.c) + t * a.c_tok);
    const T* kr = reinterpret_cast<const T*>(a.kr) + t * a.kr_tok;
    Vec<T> v[kC], x, y;
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if ((lane + 32 * i) * V < C.dc) v[i] = c[lane + 32 * i];
    if (lane < turned) {
      x = *reinterpret_cast<const Vec<T>*>(kr + lane * V);
      if (HALF) y = *reinterpret_cast<const Vec<T>*>(kr + d2 + lane * V);
    }
    __syncwarp();
    for (int i = lane; i < d2; i += 32) cs[i] = rope_cos_sin(a.tab.turn[i], slot, a.tab.mul);
    __syncwarp();
    if (page < 0 || page >= C.num_pages) {
      if (lane == 0) raise_error(a.err, ERR_PAGE, q, (uint32_t)page);
      continue;
    }
    T* dst = reinterpret_cast<T*>(const_cast<void*>(C.data)) +
             (((int64_t)page << C.log2b) + (slot & (C.b - 1))) * (C.dc + C.dr);
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if ((lane + 32 * i) * V < C.dc) reinterpret_cast<Vec<T>*>(dst)[lane + 32 * i] = v[i];
    if (lane < turned) {
      if (HALF) {
#pragma unroll
        for (int e = 0; e < V; ++e) turn_pair(x.v[e], y.v[e], cs[lane * V + e]);
        *reinterpret_cast<Vec<T>*>(dst + C.dc + d2 + lane * V) = y;
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) turn_pair(x.v[e], x.v[e + 1], cs[lane * V / 2 + e / 2]);
      }
      *reinterpret_cast<Vec<T>*>(dst + C.dc + lane * V) = x;
    }
  }
}

// The same for any strides, alignment and dims.
template <typename T>
__global__ void __launch_bounds__(256) k_append(const __grid_constant__ AppendArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)a.Q * a.rows;
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * 8) {
    const int q = (int)(t / a.rows), r = (int)(t - (int64_t)q * a.rows);
    const int ctx = a.ctx_len[q];
    const int count = a.row_count ? a.row_count[q] : a.rows;
    if (count < 0 || count > a.rows) {
      if (r == 0 && lane == 0) raise_error(a.err, ERR_ACCEPTED, q, (uint32_t)count);
      continue;
    }
    if (count == 0) continue;  // (an idle request's ctx_len is not looked at)
    if (ctx < 1 || (int64_t)ctx - 1 + count > a.max_slots) {
      if (r == 0 && lane == 0) raise_error(a.err, ERR_CTX_LEN, q, (uint32_t)ctx);
      continue;
    }
    if (r >= count) continue;
    const int slot = ctx - 1 + r;
    const LatentCache& C = a.cache;
    const int page = C.bt[(int64_t)q * C.bt_stride + (slot >> C.log2b)];
    if (page < 0 || page >= C.num_pages) {
      if (lane == 0) raise_error(a.err, ERR_PAGE, q, (uint32_t)page);
      continue;
    }
    T* dst = reinterpret_cast<T*>(const_cast<void*>(C.data)) +
             (((int64_t)page << C.log2b) + (slot & (C.b - 1))) * (C.dc + C.dr);
    const T* c = reinterpret_cast<const T*>(a.c) + t * a.c_tok;
    const T* kr = reinterpret_cast<const T*>(a.kr) + t * a.kr_tok;
    for (int i = lane; i < C.dc; i += 32) dst[i] = c[i];
    const int d2 = C.dr / 2;
    for (int i = lane; i < d2; i += 32) {
      const int e0 = a.half ? i : 2 * i, e1 = a.half ? i + d2 : 2 * i + 1;
      T v0 = kr[e0], v1 = kr[e1];
      turn_pair(v0, v1, rope_cos_sin(a.tab.turn[i], slot, a.tab.mul));
      dst[C.dc + e0] = v0;
      dst[C.dc + e1] = v1;
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int bf16, cudaStream_t s) {
  const int V = bf16 ? 8 : 4;
  const bool in_place = a.out == a.x;
  // pieces: the token's heads, their rotated part, its halves and the copied parts begin on 16 bytes
  const bool vec = (((uintptr_t)a.x | (uintptr_t)a.out) & 15) == 0 &&
                   ((a.x_tok | a.x_head | a.o_tok | a.o_head) & (V - 1)) == 0 && a.offset % V == 0 &&
                   a.head_dim % V == 0 && (a.half ? a.rope_dim / 2 : a.rope_dim) % V == 0;
  if (vec && a.tokens < (int64_t(1) << 31)) {
    const int per_head = (a.half ? a.rope_dim / 2 : a.rope_dim) / V + (in_place ? 0 : (a.head_dim - a.rope_dim) / V);
    // a whole token a block, but two blocks an SM at least where there are heads to split
    int64_t split = (2 * 148 + a.tokens - 1) / a.tokens;
    const int64_t most = std::max<int64_t>(1, (int64_t)a.heads * per_head / kRopeThreads);
    split = std::min<int64_t>(std::min(split, most), 65535);
    const int64_t need = ((int64_t)a.heads + 65534) / 65535;  // heads a block at least
    const int hpb = (int)std::max<int64_t>(need, (a.heads + split - 1) / split);
    PdlLaunch l(dim3((unsigned)a.tokens, (unsigned)((a.heads + hpb - 1) / hpb)), dim3(kRopeThreads), 0, s);
    auto kernel = bf16 ? (a.half ? k_rope_vec<__nv_bfloat16, true> : k_rope_vec<__nv_bfloat16, false>)
                       : (a.half ? k_rope_vec<float, true> : k_rope_vec<float, false>);
    return cudaLaunchKernelEx(&l.cfg, kernel, a, hpb);
  }
  const int64_t units = (int64_t)a.heads * (a.rope_dim / 2 + (in_place ? 0 : a.head_dim - a.rope_dim));
  const unsigned gx = (unsigned)(a.tokens < 148 * 8 ? a.tokens : 148 * 8);
  const int64_t gy = (units + kRopeThreads * 4 - 1) / (kRopeThreads * 4);
  PdlLaunch l(dim3(gx, (unsigned)(gy < 64 ? gy : 64)), dim3(kRopeThreads), 0, s);
  return bf16 ? cudaLaunchKernelEx(&l.cfg, k_rope_any<__nv_bfloat16>, a) : cudaLaunchKernelEx(&l.cfg, k_rope_any<float>, a);
}

cudaError_t launch_append(const AppendArgs& a, int bf16, cudaStream_t s) {
  const int V = bf16 ? 8 : 4;
  const int64_t blocks = ((int64_t)a.Q * a.rows + 7) / 8;
  PdlLaunch l(dim3((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8)), dim3(256), 0, s);
  const bool vec = (((uintptr_t)a.c | (uintptr_t)a.kr | (uintptr_t)a.cache.data) & 15) == 0 &&
                   ((a.c_tok | a.kr_tok) & (V - 1)) == 0 && (!a.half || a.cache.dr / 2 % V == 0);
  if (vec) {
    auto kernel = bf16 ? (a.half ? k_append_vec<__nv_bfloat16, true> : k_append_vec<__nv_bfloat16, false>)
                       : (a.half ? k_append_vec<float, true> : k_append_vec<float, false>);
    return cudaLaunchKernelEx(&l.cfg, kernel, a);
  }
  return bf16 ? cudaLaunchKernelEx(&l.cfg, k_append<__nv_bfloat16>, a) : cudaLaunchKernelEx(&l.cfg, k_append<float>, a);
}

}  // namespace spin
