// latent_api.cu -- host side of the latent-attention entry points
// (include/spin.h): argument checks, carving of the caller's block, rotary
// frequencies and kernel choice.  No call allocates device memory.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

#include "latent_internal.cuh"

using namespace spin;

struct spin_latent_s {
  spin_latent_config cfg;
  int device;
  int sms;
  char* base;
  ErrWord* err;
  float2* part_ml;
  float* part;
  void* kv;
  void* kr;
  int32_t* odd;
  RopeTable rope;
  void* encode_fn;  // cuTensorMapEncodeTiled
  uint32_t magic;
};

namespace {

constexpr uint32_t kMagic = 0x4c41544eu;  // "LATN"

bool alive(spin_latent lt) { return lt && lt->magic == kMagic; }

spin_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SPIN_OK;
  fprintf(stderr, "libspin: CUDA error %s\n", cudaGetErrorString(e));
  return SPIN_ECUDA;
}

// Makes the handle's device current for a call and puts the caller's back.
struct DeviceGuard {
  int before = -1;
  cudaError_t e;
  explicit DeviceGuard(int device) {
    e = cudaGetDevice(&before);
    if (e == cudaSuccess && before != device)
      e = cudaSetDevice(device);
    else
      before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};

bool eights(int x, int hi) { return x >= 8 && x <= hi && x % 8 == 0; }

// The softmax scale in log2 units, which the kernels use.
float scale_log2(const spin_latent_config* c) { return (float)((double)c->softmax_scale * 1.4426950408889634); }

bool valid_config(const spin_latent_config* c) {
  if (!c) return false;
  if (c->num_requests < 1 || c->num_requests > 16383) return false;  // Q * rows fits a grid's y
  if (c->max_slots < 1 || c->max_slots > (1 << 30)) return false;  // a tile past the last slot still fits 31 bits
  const int b = c->block_size;
  if (b < 16 || b > 256 || (b & (b - 1))) return false;
  if (c->num_heads < 1 || c->num_heads > 256) return false;
  if (!eights(c->latent_dim, 512) || !eights(c->rope_dim, kMaxRopeDim)) return false;
  if (c->topk < 1 || c->topk > 65536 || c->max_rows < 1 || c->max_rows > 4) return false;
  if (c->prefill_slots < 0 || c->prefill_slots % kSlotTile) return false;
  if (c->prefill_slots && (!eights(c->nope_dim, 256) || !eights(c->v_dim, 256))) return false;
  if (c->dtype != SPIN_F32 && c->dtype != SPIN_BF16) return false;
  if (!(c->softmax_scale > 0.0f) || !std::isfinite(scale_log2(c))) return false;
  if (c->rope_layout < SPIN_ROPE_INTERLEAVED || c->rope_layout > SPIN_ROPE_HALF) return false;
  if (c->rope_scaling < SPIN_ROPE_PLAIN || c->rope_scaling > SPIN_ROPE_YARN) return false;
  if (!(c->rope_base > 1.0) || !std::isfinite(c->rope_base)) return false;
  if (c->rope_scaling != SPIN_ROPE_PLAIN && (!(c->rope_factor >= 1.0) || !std::isfinite(c->rope_factor))) return false;
  if (c->rope_scaling == SPIN_ROPE_YARN &&
      (c->rope_original < 1 || !(c->beta_slow > 0.0f) || !(c->beta_fast > c->beta_slow) ||
       !std::isfinite(c->beta_fast) || !(c->attn_factor >= 0.0f) || !std::isfinite(c->attn_factor)))
    return false;
  if (c->reserved != 0) return false;
  // units of the flat schedule (the smaller tile) fit 31 bits
  const int64_t tiles = std::max<int64_t>(((int64_t)c->max_slots + kSimtTile - 1) / kSimtTile,
                                          (c->topk + kSimtTile - 1) / kSimtTile);
  if (tiles * c->num_requests * c->max_rows >= (int64_t(1) << 31)) return false;
  return true;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Carve {
  size_t err, turn, ml, part, kv, kr, odd, total;
};

Carve carve(const spin_latent_config* c) {
  Carve k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  const size_t el = c->dtype == SPIN_BF16 ? 2 : 4;
  // two shares for each block; of the two kernels' needs the larger.  A
  // block of either takes at most its group's heads, and the last group may
  // hold fewer heads than its slots.
  const int group = std::min(kTcHeads, (c->num_heads + 15) / 16 * 16);
  const size_t heads = std::max<size_t>((size_t)2 * kTcBlocks * group, (size_t)2 * kSimtBlocks * kSimtHeads);
  // (the expanded form's parts take the same place: 256 rows of each of 148 blocks)
  const size_t parts = c->prefill_slots ? (size_t)kTcBlocks * 256 : 0;
  k.err = take(sizeof(ErrWord));
  k.turn = take(kMaxRopeDim / 2 * sizeof(uint64_t));
  k.ml = take(std::max(heads, parts) * sizeof(float2));
  k.part = take(std::max(heads * c->latent_dim, parts * c->v_dim) * sizeof(float));
  k.kv = take(c->prefill_slots ? (size_t)c->prefill_slots * c->num_heads * (c->nope_dim + c->v_dim) * el : 0);
  k.kr = take(c->prefill_slots ? (size_t)c->prefill_slots * c->rope_dim * el : 0);
  k.odd = take(c->prefill_slots ? (size_t)c->prefill_slots / kSlotTile * c->num_heads * sizeof(int32_t) : 0);
  k.total = off;
  return k;
}

// f_i of every pair in double (arXiv 2309.00071 for YaRN), as the fraction of
// a turn per position in units of 2^-64.
struct RopeValues {
  uint64_t turn[kMaxRopeDim / 2];
  float mul;
};
RopeValues rope_values(const spin_latent_config& c) {
  RopeValues t{};
  const int d = c.rope_dim;
  const double two_pi = 6.283185307179586476925286766559;
  t.mul = 1.0f;
  double lo = 0, hi = 0;
  if (c.rope_scaling == SPIN_ROPE_YARN) {
    // the pair that turns `turns` times within rope_original positions
    auto pair_of = [&](double turns) {
      return d * std::log(c.rope_original / (turns * two_pi)) / (2.0 * std::log(c.rope_base));
    };
    lo = std::max(std::floor(pair_of(c.beta_fast)), 0.0);
    hi = std::min(std::ceil(pair_of(c.beta_slow)), (double)(d - 1));
    t.mul = c.attn_factor > 0.0f ? c.attn_factor : (float)(0.1 * std::log(c.rope_factor) + 1.0);
  }
  for (int i = 0; i < d / 2; ++i) {
    double f = std::pow(c.rope_base, -2.0 * i / d);
    if (c.rope_scaling == SPIN_ROPE_LINEAR) f /= c.rope_factor;
    if (c.rope_scaling == SPIN_ROPE_YARN) {
      const double g = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      f = f / c.rope_factor * g + f * (1.0 - g);
    }
    const long double turn = (long double)f / 6.283185307179586476925286766559005768L;  // f <= 1: below 1/6 of a turn
    t.turn[i] = (uint64_t)std::llroundl(turn * 18446744073709551616.0L);
  }
  return t;
}

LatentCache cache_of(spin_latent lt, const void* cache, int32_t num_pages, const int32_t* bt, int32_t bt_stride) {
  LatentCache c;
  c.data = cache;
  c.bt = bt;
  c.num_pages = num_pages;
  c.bt_stride = bt_stride;
  c.b = lt->cfg.block_size;
  c.log2b = 0;
  while ((1 << c.log2b) < c.b) ++c.log2b;
  c.dc = lt->cfg.latent_dim;
  c.dr = lt->cfg.rope_dim;
  return c;
}

// The block table must cover every slot that a valid ctx_len can name.
bool cache_ok(spin_latent lt, const void* cache, int32_t num_pages, const int32_t* bt, int32_t bt_stride) {
  const int64_t blocks = ((int64_t)lt->cfg.max_slots + lt->cfg.block_size - 1) / lt->cfg.block_size;
  return cache && num_pages >= 1 && bt && bt_stride >= blocks;
}

}  // namespace

extern "C" {

size_t spin_latent_bytes(const spin_latent_config* cfg) { return valid_config(cfg) ? carve(cfg).total : 0; }

spin_status spin_latent_create(const spin_latent_config* cfg, void* dev_mem, size_t bytes, spin_stream_t stream,
                               spin_latent* out) {
  if (!out) return SPIN_EINVAL;
  *out = nullptr;
  if (!valid_config(cfg) || !dev_mem || ((uintptr_t)dev_mem & 255)) return SPIN_EINVAL;
  const Carve k = carve(cfg);
  if (bytes < k.total) return SPIN_ENOMEM;
  cudaPointerAttributes at{};
  cudaError_t e = cudaPointerGetAttributes(&at, dev_mem);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_status(e);
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return SPIN_EINVAL;
  DeviceGuard guard(at.device);
  if (guard.e != cudaSuccess) return cuda_status(guard.e);
  spin_latent lt = new (std::nothrow) spin_latent_s();
  if (!lt) return SPIN_ENOMEM;
  lt->cfg = *cfg;
  lt->device = at.device;
  lt->base = (char*)dev_mem;
  lt->err = (ErrWord*)(lt->base + k.err);
  lt->part_ml = (float2*)(lt->base + k.ml);
  lt->part = (float*)(lt->base + k.part);
  lt->kv = lt->base + k.kv;
  lt->kr = lt->base + k.kr;
  lt->odd = (int32_t*)(lt->base + k.odd);
  const RopeValues rope = rope_values(*cfg);
  lt->rope.turn = (const uint64_t*)(lt->base + k.turn);
  lt->rope.mul = rope.mul;
  lt->sms = kTcBlocks;
  cudaDeviceGetAttribute(&lt->sms, cudaDevAttrMultiProcessorCount, at.device);
  cudaDriverEntryPointQueryResult qres;
  void* fn = nullptr;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &qres) == cudaSuccess &&
      qres == cudaDriverEntryPointSuccess)
    lt->encode_fn = fn;
  cudaGetLastError();
  e = cudaMemsetAsync(lt->err, 0, sizeof(ErrWord), (cudaStream_t)stream);
  // (from pageable memory: copied out of `rope` before the call returns)
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(lt->base + k.turn, rope.turn, sizeof(rope.turn), cudaMemcpyHostToDevice, (cudaStream_t)stream);
  if (e == cudaSuccess) e = prepare_attn_tc();
  if (e == cudaSuccess) e = prepare_attn_simt();
  if (e == cudaSuccess) e = prepare_prefill_tc();
  if (e != cudaSuccess) {
    delete lt;
    return cuda_status(e);
  }
  lt->magic = kMagic;
  *out = lt;
  return SPIN_OK;
}

spin_status spin_latent_destroy(spin_latent lt) {
  if (!alive(lt)) return SPIN_ESTATE;
  lt->magic = 0;
  delete lt;
  return SPIN_OK;
}

spin_status spin_rope(spin_latent lt, int64_t tokens, int heads, int head_dim, int offset, const void* x,
                      int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions_dev, void* out,
                      int64_t out_token_stride, int64_t out_head_stride, spin_stream_t stream) {
  if (!alive(lt)) return SPIN_ESTATE;
  const spin_latent_config& c = lt->cfg;
  if (tokens < 0 || heads < 1 || head_dim < c.rope_dim || offset < 0 || offset > head_dim - c.rope_dim)
    return SPIN_EINVAL;
  if ((int64_t)heads * head_dim > (int64_t(1) << 30)) return SPIN_EINVAL;  // 32-bit element counts, and a step on
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0) return SPIN_EINVAL;
  if (tokens == 0) return SPIN_OK;
  if (!x || !out || !positions_dev) return SPIN_EINVAL;
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride)) return SPIN_EINVAL;
  DeviceGuard guard(lt->device);
  if (guard.e != cudaSuccess) return cuda_status(guard.e);
  RopeArgs a{lt->rope, tokens,        heads,         head_dim,      offset, c.rope_dim,       c.rope_layout == SPIN_ROPE_HALF,
             x,        x_token_stride, x_head_stride, positions_dev, out,    out_token_stride, out_head_stride};
  return cuda_status(launch_rope(a, c.dtype == SPIN_BF16, (cudaStream_t)stream));
}

spin_status spin_latent_append(spin_latent lt, int rows, const void* c_dev, int64_t c_token_stride,
                               const void* kr_dev, int64_t kr_token_stride, void* cache, int32_t num_pages,
                               const int32_t* block_table, int32_t bt_stride, const int32_t* ctx_len_dev,
                               const int32_t* row_count_dev, spin_stream_t stream) {
  if (!alive(lt)) return SPIN_ESTATE;
  const spin_latent_config& c = lt->cfg;
  if (rows < 1 || c_token_stride < 0 || kr_token_stride < 0 || !c_dev || !kr_dev || !ctx_len_dev ||
      !cache_ok(lt, cache, num_pages, block_table, bt_stride))
    return SPIN_EINVAL;
  DeviceGuard guard(lt->device);
  if (guard.e != cudaSuccess) return cuda_status(guard.e);
  AppendArgs a{};
  a.tab = lt->rope;
  a.cache = cache_of(lt, cache, num_pages, block_table, bt_stride);
  a.Q = c.num_requests;
  a.rows = rows;
  a.half = c.rope_layout == SPIN_ROPE_HALF;
  a.max_slots = c.max_slots;
  a.c = c_dev;
  a.kr = kr_dev;
  a.c_tok = c_token_stride;
  a.kr_tok = kr_token_stride;
  a.ctx_len = ctx_len_dev;
  a.row_count = row_count_dev;
  a.err = lt->err;
  return cuda_status(launch_append(a, c.dtype == SPIN_BF16, (cudaStream_t)stream));
}

spin_status spin_latent_attention(spin_latent lt, int rows, const void* cache, int32_t num_pages,
                                  const int32_t* block_table, int32_t bt_stride, const void* q_latent,
                                  int64_t ql_token_stride, int64_t ql_head_stride, const void* q_rope,
                                  int64_t qr_token_stride, int64_t qr_head_stride, const int32_t* ctx_len_dev,
                                  const int32_t* topk_dev, void* out, float* lse, spin_stream_t stream) {
  if (!alive(lt)) return SPIN_ESTATE;
  const spin_latent_config& c = lt->cfg;
  if (rows < 1 || rows > c.max_rows || ql_token_stride < 0 || ql_head_stride < 0 || qr_token_stride < 0 ||
      qr_head_stride < 0 || !q_latent || !q_rope || !ctx_len_dev || !out ||
      !cache_ok(lt, cache, num_pages, block_table, bt_stride))
    return SPIN_EINVAL;
  DeviceGuard guard(lt->device);
  if (guard.e != cudaSuccess) return cuda_status(guard.e);
  AttnArgs a{};
  a.cache = cache_of(lt, cache, num_pages, block_table, bt_stride);
  a.Q = c.num_requests;
  a.rows = rows;
  a.H = c.num_heads;
  a.max_slots = c.max_slots;
  a.topk = c.topk;
  a.list = topk_dev;
  a.ctx_len = ctx_len_dev;
  a.ql = q_latent;
  a.qr = q_rope;
  a.ql_tok = ql_token_stride;
  a.ql_head = ql_head_stride;
  a.qr_tok = qr_token_stride;
  a.qr_head = qr_head_stride;
  const int64_t per16 = c.dtype == SPIN_BF16 ? 8 : 4;
  a.q_vec = ((uintptr_t)q_latent & 15) == 0 && ((uintptr_t)q_rope & 15) == 0 && ql_token_stride % per16 == 0 &&
            ql_head_stride % per16 == 0 && qr_token_stride % per16 == 0 && qr_head_stride % per16 == 0;
  a.scale_log2 = scale_log2(&c);
  a.out = out;
  a.lse = lse;
  a.err = lt->err;
  a.part = lt->part;
  a.part_ml = lt->part_ml;
  const int bf16 = c.dtype == SPIN_BF16;
  // items * tiles bounds the units, and more blocks than units have nothing to do
  auto plan = [&](int tile, int group, int blocks) {
    a.tile = tile;
    a.group = group;
    a.ngroups = (a.H + group - 1) / group;
    const int64_t n = a.list ? a.topk : a.max_slots;
    a.ranges = (int)std::min<int64_t>(std::max(1, blocks / a.ngroups), (int64_t)a.Q * rows * ((n + tile - 1) / tile));
    a.whole = 0;
    a.rest = a.ranges;
    a.per = (a.topk + tile - 1) / tile;
    a.total = a.Q * rows * a.per;
  };
  cudaError_t e;
  if (attn_tc_supported(a, bf16)) {
    const int groups = (a.H + kTcHeads - 1) / kTcHeads;
    plan(kTcTile, ((a.H + groups - 1) / groups + 15) / 16 * 16, std::min(lt->sms, kTcBlocks));
    if (a.list) {
      // Equally long items: as many whole ones as go round, then the others
      //   a block each,
      //   or cut evenly, `cut` blocks each (the join costs about as much as 2 tiles),
      //   or as one run of units over all blocks (and blocks that change items, about 5 tiles),
      // whichever ends first.  128 items of 32 tiles on 148 blocks: 73 us as one run, 61 us a block each.
      const int items = a.Q * rows, per = a.per;
      a.whole = items / a.ranges;
      const int left = items - a.whole * a.ranges;
      if (left) {
        const int cut = std::min(a.ranges / left, per);
        const int even = cut > 1 ? (per + cut - 1) / cut + 2 : per;
        const int run = (int)((int64_t)left * per / a.ranges) + 5;
        if (even <= run) a.rest = left * cut;
        if (a.rest == left && a.whole == 0) {  // a block each
          a.ranges = left;
          a.whole = 1;
        }
        a.total = (items - a.whole * a.ranges) * per;
      } else {
        a.total = 0;
      }
    }
    e = launch_attn_tc(a, (cudaStream_t)stream);
  } else {
    plan(kSimtTile, kSimtHeads, std::min(2 * lt->sms, kSimtBlocks));
    e = launch_attn_simt(a, bf16, (cudaStream_t)stream);
  }
  const int left = a.Q * rows - a.whole * a.ranges;  // items that may lie in several blocks' ranges
  if (e == cudaSuccess && left && !(a.list && a.rest == left)) e = launch_attn_combine(a, bf16, (cudaStream_t)stream);
  return cuda_status(e);
}

spin_status spin_latent_prefill(spin_latent lt, int rows, const void* cache, int32_t num_pages,
                                const int32_t* block_table, int32_t bt_stride, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, const void* w_kv, const int32_t* ctx_len_dev,
                                const int32_t* row_count_dev, void* out, spin_stream_t stream) {
  if (!alive(lt)) return SPIN_ESTATE;
  const spin_latent_config& c = lt->cfg;
  if (rows < 1 || q_token_stride < 0 || q_head_stride < 0 || !q || !w_kv || !ctx_len_dev || !out ||
      !cache_ok(lt, cache, num_pages, block_table, bt_stride))
    return SPIN_EINVAL;
  if (!c.prefill_slots) return SPIN_EUNSUPPORTED;
  // blocks of the launch: 256 rows of a head each
  if (rows > (1 << 30) || ((int64_t)rows + 255) / 256 * c.num_requests * c.num_heads >= (int64_t(1) << 31) - kTcBlocks)
    return SPIN_EUNSUPPORTED;
  DeviceGuard guard(lt->device);
  if (guard.e != cudaSuccess) return cuda_status(guard.e);
  PrefillArgs a{};
  a.cache = cache_of(lt, cache, num_pages, block_table, bt_stride);
  a.Q = c.num_requests;
  a.rows = rows;
  a.H = c.num_heads;
  a.dn = c.nope_dim;
  a.dv = c.v_dim;
  a.max_slots = c.max_slots;
  a.cap = c.prefill_slots;
  a.ctx_len = ctx_len_dev;
  a.row_count = row_count_dev;
  a.q = q;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.w = w_kv;
  a.out = out;
  a.kv = lt->kv;
  a.kr = lt->kr;
  a.odd = lt->odd;
  a.part = lt->part;
  a.part_ml = lt->part_ml;
  a.scale_log2 = scale_log2(&c);
  a.err = lt->err;
  const int bf16 = c.dtype == SPIN_BF16;
  const int64_t per16 = bf16 ? 8 : 4;
  a.q_vec = ((uintptr_t)q & 15) == 0 && q_token_stride % per16 == 0 && q_head_stride % per16 == 0;
  if (lt->encode_fn && prefill_tc_supported(a, bf16))
    return cuda_status(launch_prefill_tc(a, lt->encode_fn, lt->sms, (cudaStream_t)stream));
  cudaError_t e = launch_expand_simt(a, bf16, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_prefill_simt(a, bf16, (cudaStream_t)stream);
  return cuda_status(e);
}

spin_status spin_latent_error(spin_latent lt, spin_stream_t stream, uint32_t* word_out) {
  if (!alive(lt)) return SPIN_ESTATE;
  DeviceGuard guard(lt->device);
  cudaStream_t s = (cudaStream_t)stream;
  ErrWord h{};
  cudaError_t e = guard.e;
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&h, lt->err, sizeof(ErrWord), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(lt->err, 0, sizeof(ErrWord), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e);
  if (word_out) *word_out = h.flags;
  if (h.flags & ERR_TIMEOUT) return SPIN_ETIMEOUT;
  return h.flags ? SPIN_EDEVICE : SPIN_OK;
}

}  // extern "C"
