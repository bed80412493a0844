// k_rope.cu -- rotary positions, and the append of new tokens to the paged
// latent cache.
//
// A pair (x, y) of a head turns by the angle t of its position:
//   (x cos t - y sin t, x sin t + y cos t),
// computed in fp32 from the stored values and rounded once.  Both kernels
// move each byte once and compute little: they are bound by HBM, and at
// decode sizes by the latency of one dependent load (position), the sine and
// the store.
#include "latent_internal.cuh"

namespace spin {
namespace {

constexpr int kRopeThreads = 256;

template <typename T>
__device__ __forceinline__ void turn_pair(T& x, T& y, float2 cs) {
  const float a = to_f32(x), b = to_f32(y);
  x = from_f32<T>(a * cs.x - b * cs.y);
  y = from_f32<T>(a * cs.y + b * cs.x);
}

// One element pair or one copied element per thread and step: any strides,
// alignment and dims.
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

// New tokens into the cache: one warp per token.
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
  const int64_t units = (int64_t)a.heads * (a.rope_dim / 2 + (a.out == a.x ? 0 : a.head_dim - a.rope_dim));
  const unsigned gx = (unsigned)(a.tokens < 148 * 8 ? a.tokens : 148 * 8);
  const int64_t gy = (units + kRopeThreads * 4 - 1) / (kRopeThreads * 4);
  PdlLaunch l(dim3(gx, (unsigned)(gy < 64 ? gy : 64)), dim3(kRopeThreads), 0, s);
  return bf16 ? cudaLaunchKernelEx(&l.cfg, k_rope_any<__nv_bfloat16>, a) : cudaLaunchKernelEx(&l.cfg, k_rope_any<float>, a);
}

cudaError_t launch_append(const AppendArgs& a, int bf16, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.Q * a.rows + 7) / 8;
  PdlLaunch l(dim3((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8)), dim3(256), 0, s);
  return bf16 ? cudaLaunchKernelEx(&l.cfg, k_append<__nv_bfloat16>, a) : cudaLaunchKernelEx(&l.cfg, k_append<float>, a);
}

}  // namespace spin
