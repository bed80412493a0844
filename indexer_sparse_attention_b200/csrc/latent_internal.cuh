// latent_internal.cuh -- arguments and device helpers shared by the latent
// attention kernels (rotary positions, cache append, absorbed and expanded
// attention).  Nothing here is part of the C ABI.
#pragma once

#include "block_scan.cuh"
#include "spin_internal.cuh"

namespace spin {

// ---------------------------------------------------------------------------
// Rotary angles.  The turn of pair i at position p is p * f_i / (2 pi), of
// which only the fraction matters.  With F_i = round(2^64 * frac(f_i / (2
// pi))) the fraction is p * F_i modulo 2^64: one integer product, wrong by at
// most |p| * 2^-65 of a turn beside f_i's own rounding (a double: |p| * f_i *
// 2^-51 radians at most), at every position and either sign, where an angle in
// 32-bit floats loses about 2^-24 of p * f_i itself.  The fraction as a float
// costs up to 2^-26 of a turn, half a step of the largest ones.
// ---------------------------------------------------------------------------
constexpr int kMaxRopeDim = 128;
struct RopeTable {
  const uint64_t* turn;  // [rope_dim / 2] in device memory (each thread reads another pair's)
  float mul;             // on cos and sin
};

// cos and sin of a position, scaled.  The fraction's top 32 bits, read as a
// signed number of 2^-31 half turns, go to sincospi.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turn, int32_t pos, float mul) {
  const uint64_t frac = (uint64_t)(int64_t)pos * turn;
  const float half_turns = (float)(int32_t)(frac >> 32) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * mul, s * mul);
}

// ---------------------------------------------------------------------------
// Element types
// ---------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

struct RopeArgs {
  RopeTable tab;
  int64_t tokens;
  int heads, head_dim, offset, rope_dim, half;
  const void* x;
  int64_t x_tok, x_head;
  const int32_t* pos;
  void* out;
  int64_t o_tok, o_head;
};
cudaError_t launch_rope(const RopeArgs& a, int bf16, cudaStream_t s);

// The paged latent cache and where a request's slots lie in it.
struct LatentCache {
  const void* data;  // [num_pages][b][dc + dr]
  const int32_t* bt;
  int32_t num_pages, bt_stride;
  int b, log2b;
  int dc, dr;
};

struct AppendArgs {
  RopeTable tab;
  LatentCache cache;
  int Q, rows, half;
  int32_t max_slots;
  const void* c;
  const void* kr;
  int64_t c_tok, kr_tok;
  const int32_t* ctx_len;
  const int32_t* row_count;
  ErrWord* err;
};
cudaError_t launch_append(const AppendArgs& a, int bf16, cudaStream_t s);

// ---------------------------------------------------------------------------
// Absorbed attention: flat schedule.  An item is one (request, row); its
// tokens are cut into tiles, at least one per item.  All items' tiles in a
// row are the units; of the blocks that serve one group of heads (`ranges` of
// them, or as many as there are units) block u takes units [U u / ranges, U
// (u + 1) / ranges), so ragged contexts and few rows fill the SMs alike.  An item that lies in one block's range is
// finished there.  Else each block leaves its share -- maximum, sum and
// unnormalised output, in fp32 -- in one of its two slots of the workspace
// (slot 0: the item that holds the block's first unit, slot 1: the item that
// runs on past its last), and the combine kernel joins the shares in block
// order, so the result does not depend on timing.  Lists make all items
// equally long: there each block takes `whole` items whole before its range
// of the other items' units, which halves what is left as shares.
// ---------------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  LatentCache cache;
  int Q, rows, H;
  int32_t max_slots;
  int topk;                  // entries of a list
  const int32_t* list;       // [Q][rows][topk] or null
  const int32_t* ctx_len;
  const void* ql;
  const void* qr;
  int64_t ql_tok, ql_head, qr_tok, qr_head;
  int q_vec;                 // every head of ql and qr starts on 16 bytes
  float scale_log2;          // softmax scale * log2(e)
  void* out;                 // [Q][rows][H][dc]
  float* lse;                // [Q][rows][H] or null
  ErrWord* err;
  int tile;                  // tokens of a tile
  int group;                 // heads of a block
  int ngroups;               // ceil(H / group)
  int ranges;                // blocks per head group, at most
  int whole;                 // items that each block takes whole (lists only)
  int rest;                  // of the blocks, those that share the other items, at most
  int per;                   // lists: tiles of an item, and of the items that are not taken whole
  int total;
  float* part;               // [ngroups * ranges * 2][group][dc] unnormalised outputs
  float2* part_ml;           // [ngroups * ranges * 2][group] (maximum in log2 units, sum)
};

// The last slot + 1 that row r of request q may attend to (0: its ctx_len is
// out of range), and the number of tiles of the item.
__device__ __forceinline__ int attn_end_at(const AttnArgs& a, int ctx, int r) {
  return (ctx >= 1 && (int64_t)ctx + a.rows - 1 <= a.max_slots) ? ctx + r : 0;
}
__device__ __forceinline__ int attn_end(const AttnArgs& a, int q, int r) { return attn_end_at(a, a.ctx_len[q], r); }
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, int end) {
  if (a.list) return a.per;
  return end > 0 ? (end + a.tile - 1) / a.tile : 1;
}

// First unit of range u of `ranges` over `total` >= ranges units, and the
// range that holds unit g.  (A division of 64 bits takes hundreds of cycles; most
// products fit 32.)
__device__ __forceinline__ int div_units(uint64_t n, int d) {
  return n >> 32 ? (int)(n / (uint32_t)d) : (int)((uint32_t)n / (uint32_t)d);
}
__device__ __forceinline__ int range_begin(int total, int ranges, int u) {
  return div_units((uint64_t)total * (uint32_t)u, ranges);
}
__device__ __forceinline__ int range_of(int total, int ranges, int g) {
  // begin(u) <= g  <=>  total u < (g + 1) ranges
  return div_units((uint64_t)(g + 1) * (uint32_t)ranges - 1, total);
}

// The units of the items that are not taken whole: how many there are and over
// how many ranges they go, the item asked for and its first unit.
struct Place {
  int total, ranges;
  int item, first;
};

// Places either `item`, or (item < 0) the item that holds the first unit of
// range u (item 0 where there is no such range).  All threads of the block; tmp:
// 36 ints of shared memory.  The host has checked that all units together fit
// 31 bits.
__device__ __forceinline__ Place attn_place(const AttnArgs& a, int item, int u, int* tmp) {
  const int items = a.Q * a.rows;
  Place p;
  if (a.list) {
    const int base = a.whole * a.ranges;
    p.total = a.total;
    p.ranges = min(a.rest, a.total);
    const int i = item >= 0 ? item - base : u < p.ranges ? range_begin(p.total, p.ranges, u) / a.per : 0;
    p.item = base + i;
    p.first = i * a.per;
    return p;
  }
  // every item's tiles, one after the other
  auto tiles = [&](int i) { return i < items ? attn_tiles(a, attn_end(a, i / a.rows, i % a.rows)) : 0; };
  if (items <= 128) {
    // each warp by itself, four items a lane: no barriers
    const int lane = threadIdx.x & 31;
    int n[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += n[k] = tiles(4 * lane + k);
    const int up = warp_inclusive_scan(sum);
    p.total = __shfl_sync(0xffffffffu, up, 31);
    p.ranges = min(a.rest, p.total);
    const int want = item >= 0 || u >= p.ranges ? 0 : range_begin(p.total, p.ranges, u);
    int at = up - sum, here = -1, start = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (item >= 0 ? 4 * lane + k == item : at <= want && want < at + n[k]) {
        here = 4 * lane + k;
        start = at;
      }
      at += n[k];
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here >= 0)) - 1;
    p.item = __shfl_sync(0xffffffffu, here, src);
    p.first = __shfl_sync(0xffffffffu, start, src);
    return p;
  }
  int sum = 0;
  for (int i = threadIdx.x; i < items; i += blockDim.x) sum += tiles(i);
  block_exclusive_scan(sum, tmp, &p.total);
  p.ranges = min(a.rest, p.total);
  const int want = item >= 0 || u >= p.ranges ? 0 : range_begin(p.total, p.ranges, u);
  int carry = 0;
  for (int base = 0; base < items; base += blockDim.x) {
    const int i = base + (int)threadIdx.x, m = tiles(i);
    int tot;
    const int at = carry + block_exclusive_scan(m, tmp, &tot);
    if (item >= 0 ? i == item : at <= want && want < at + m) {
      tmp[33] = i;
      tmp[34] = at;
    }
    carry += tot;
    if (item >= 0 ? base + (int)blockDim.x > item : carry > want) break;
  }
  __syncthreads();
  p.item = tmp[33];
  p.first = tmp[34];
  __syncthreads();
  return p;
}

// Cache row (page * b + place) of a slot, or -1 where the slot is not one
// that the row attends to or its page lies outside the cache.
__device__ __forceinline__ int64_t cache_row(const LatentCache& c, int q, int slot, ErrWord* err) {
  const int page = c.bt[(int64_t)q * c.bt_stride + (slot >> c.log2b)];
  if (page < 0 || page >= c.num_pages) {
    raise_error(err, ERR_PAGE, q, (uint32_t)page);
    return -1;
  }
  return ((int64_t)page << c.log2b) + (slot & (c.b - 1));
}

// Heads and tokens of a block of the simple kernel, and its grid limit.
constexpr int kSimtHeads = 8, kSimtTile = 32, kSimtBlocks = 296;
// Heads, tokens and grid limit of the tensor-core kernel (one block per SM).
constexpr int kTcHeads = 64, kTcTile = 64, kTcBlocks = 148;

// The prepare_ calls raise the kernels' shared-memory limits on the current
// device, once for each handle.
cudaError_t prepare_attn_simt();
cudaError_t prepare_attn_tc();
cudaError_t prepare_prefill_tc();
cudaError_t launch_attn_simt(const AttnArgs& a, int bf16, cudaStream_t s);
bool attn_tc_supported(const AttnArgs& a, int bf16);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_combine(const AttnArgs& a, int bf16, cudaStream_t s);

// ---------------------------------------------------------------------------
// Expanded attention.  Each request's slots 0 .. end - 1 (end = ctx_len - 1 +
// row_count) are expanded into rows off .. off + end - 1 of the workspace,
// off the sum of the earlier requests' ends, each rounded up to kSlotTile.
// ---------------------------------------------------------------------------
constexpr int kSlotTile = 128;

struct PrefillArgs {
  LatentCache cache;
  int Q, rows, H, dn, dv;
  int32_t max_slots;
  int64_t cap;               // workspace rows
  const int32_t* ctx_len;
  const int32_t* row_count;  // or null
  const void* q;             // [Q][rows][H][dn + dr]
  int64_t q_tok, q_head;
  int q_vec;                 // every head of q starts on 16 bytes
  const void* w;             // [H][dn + dv][dc]
  void* out;                 // [Q][rows][H][dv]
  void* kv;                  // [H][cap][dn + dv]
  void* kr;                  // [cap][dr]
  int32_t* odd;              // tensor-core kernel: [H][cap / 128], a tile's first slot with values that are not finite
  float* part;               // tensor-core kernel: parts cut along the keys, [148][256][dv]
  float2* part_ml;           // [148][256] (maximum in log2 units, sum)
  int planned;               // tensor-core kernel: few enough rows to rank and cut
  float scale_log2;
  ErrWord* err;
};

// The rows of a request that are computed (0: none, or its lengths are out of
// range) and the slots its last row sees.
struct Chunk {
  int ctx, count, end;
};
__device__ __forceinline__ Chunk prefill_chunk(const PrefillArgs& a, int q, bool report) {
  Chunk c;
  c.ctx = a.ctx_len[q];
  c.count = a.row_count ? a.row_count[q] : a.rows;
  if (c.count < 0 || c.count > a.rows) {
    if (report) raise_error(a.err, ERR_ACCEPTED, q, (uint32_t)c.count);
    c.count = 0;
  } else if (c.count && (c.ctx < 1 || (int64_t)c.ctx - 1 + c.count > a.max_slots)) {
    if (report) raise_error(a.err, ERR_CTX_LEN, q, (uint32_t)c.ctx);
    c.count = 0;
  }
  c.end = c.count ? c.ctx - 1 + c.count : 0;
  return c;
}

// Workspace rows before request q (`tmp`: 33 int64 of shared memory; all
// threads of the block).
__device__ __forceinline__ int64_t prefill_rows_before(const PrefillArgs& a, int q, int64_t* tmp) {
  int64_t sum = 0;
  for (int i = threadIdx.x; i < q; i += blockDim.x)
    sum += (prefill_chunk(a, i, false).end + kSlotTile - 1) / kSlotTile * kSlotTile;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0;
  for (int w = 0; w < (int)(blockDim.x + 31) / 32; ++w) sum += tmp[w];
  __syncthreads();
  return sum;
}

bool prefill_tc_supported(const PrefillArgs& a, int bf16);
cudaError_t launch_prefill_tc(const PrefillArgs& a, void* encode_fn, int sms, cudaStream_t s);
cudaError_t launch_expand_simt(const PrefillArgs& a, int bf16, cudaStream_t s);
cudaError_t launch_prefill_simt(const PrefillArgs& a, int bf16, cudaStream_t s);

}  // namespace spin
