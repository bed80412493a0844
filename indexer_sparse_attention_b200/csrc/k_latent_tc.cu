// k_latent_tc.cu -- absorbed latent attention on the 5th-generation tensor
// cores: bf16, latent width 512, rotary width 64.
//
// For one (request, row) and a group of NH <= 64 heads a block runs over
// tiles of 64 tokens, each token's cache entry [c | kr] (1152 bytes) read
// once into shared memory and used by both products:
//   S  [heads 64 x tokens 64] = Q [heads x 576] . K^T     M 64,  N 64, K 576
//   O^T[512 x heads]         += C^T [512 x tokens] . P^T  M 128 x 4, N NH, K 64
// C^T is the very tile that K is (an MN-major view of it), so a token crosses
// L2 -> SM once per 64 heads.  The second product is transposed because its
// fp32 accumulator is the largest thing here: with heads as N it takes 4 NH
// of the 512 TMEM columns for any number of heads, where heads as M would
// take all 512 at every head count and leave none for S.
//
// Running softmax with a lazy reference: weights are 2^(s - m) for a
// reference m that is moved (and O, l rescaled) only where a row's maximum has
// grown by more than 8 (log2 units), so O is almost never touched between
// products; weights stay below 2^8, sums and O are fp32.  The weights are
// rounded to bf16 for the second product (half a step, 2^-8 of each weight, is
// what the outputs' own rounding costs as well); their sum is of the
// unrounded ones.
//
// Warps (384 threads, one block per SM):
//   0..3  softmax: S from TMEM (warp w: heads 16 w .. 16 w + 15), weights to
//         shared memory; at an item's end O^T from TMEM to the output or to the
//         block's share
//   4..7  producers: list entries -> cache rows (looked up two tiles ahead)
//         -> 16-byte asynchronous copies, eight lanes a 128-byte line.  A
//         gather by TMA (four rows a request) moved 2.0 TB/s from one warp's
//         lanes and 4.3 TB/s from four warps, these copies 6.45 TB/s (64 rows of
//         1152 bytes at random from 302 MB, 148 blocks)
//   8, 9  issue of the first and of the second product
//   10, 11 Q tile of the next item into shared memory
// Two 72 KB token tiles in flight, each cut into five parts (the rotary part
// and four of 128 latent columns) with their own barriers: a part is
// reloaded as soon as the second product has read its columns, and S starts
// on the parts that have landed.
#include <algorithm>

#include "latent_internal.cuh"
#include "umma.cuh"

namespace spin {
namespace {

using namespace umma;

constexpr int kDC = 512, kDR = 64, kW = kDC + kDR;
constexpr int kTok = kTcTile;                    // tokens of a tile
constexpr int kBlk = kTok * 128;                 // bytes of a 64-column block of a tile
constexpr int kBlocks = kW / 64;                 // 9: 8 of c, then kr
constexpr int kStageBytes = kBlocks * kBlk;
constexpr int kStages = 2;
constexpr int kParts = 5;                        // 0..3: column blocks 2 p, 2 p + 1; 4: kr
constexpr int kInfo = 4;                         // ring of tile infos
constexpr int kThreads = 384;
constexpr int kProducers = 128, kMmaWarp = 8, kQThreads = 64;
constexpr float kLazy = 8.0f;
constexpr uint32_t kSCol = 256;                  // S buffers behind O^T's 4 * 64 columns
constexpr uint32_t kTmemCols = 512;

struct Info {
  uint32_t even, odd;  // the even and the odd tokens that are attended to
  int flags;           // 1: first tile of an item's share, 2: its last, 4: the block's last
};

struct Bars {
  uint64_t full[kStages][kParts];   // copies landed
  uint64_t empty[kStages][kParts];  // MMAs that read the part
  uint64_t info[kInfo];             // producer: tile info written
  uint64_t sfull[2];                // S complete
  uint64_t sfree[2];                // S read
  uint64_t pfull;                   // weights written, O rescaled
  uint64_t pempty;                  // second product complete
  uint64_t qfull, qempty;
  uint64_t oempty;                  // O^T read out
  uint64_t done[2];
};

struct Misc {
  Bars bars;
  Info info[kInfo];
  alignas(16) float fac[kTcHeads];  // rescale factors, then 1 / sum
  int tmp[35];
  uint32_t tmem;
  int abort_flag;
};

__host__ __device__ constexpr uint32_t smem_bytes(int nh) {
  return 1024 + (uint32_t)(kBlocks * nh * 128 + kStages * kStageBytes + nh * 128) + (uint32_t)sizeof(Misc);
}
static_assert(smem_bytes(kTcHeads) <= 227 * 1024, "one block's shared memory");

// The walk over a block's shares of items: units [at, stop).
struct Walk {
  int item, first, at, stop;
  int q, r, end, n, t0, t1;
  __device__ __forceinline__ void open(const AttnArgs& a) {
    q = item / a.rows;
    r = item - q * a.rows;
    end = attn_end(a, q, r);
    n = attn_tiles(a, end);
    t0 = at - first;
    t1 = min(n, stop - first);
  }
  __device__ __forceinline__ bool next() {  // false: nothing left
    at = first + t1;
    first += n;
    ++item;
    return at < stop;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a) {
  pdl_enter();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NH = a.group, H = a.H;
  // Q first: the M = 64 rows of S's A operand run past the NH rows of a
  // block of Q into what follows (rows that nothing reads)
  uint8_t* q_sm = smem;
  uint8_t* kv_sm = q_sm + kBlocks * NH * 128;
  uint8_t* p_sm = kv_sm + kStages * kStageBytes;
  Misc& ms = *reinterpret_cast<Misc*>(p_sm + NH * 128);
  const uint32_t q_at = smem_u32(q_sm), kv_at = smem_u32(kv_sm), p_at = smem_u32(p_sm);
  Bars& B = ms.bars;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const Ctl ctl{&ms.abort_flag, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x % a.ngroups, u = blockIdx.x / a.ngroups;
  const int h0 = g * NH;

  // the block's units (all threads)
  const int total = attn_units_before(a, a.Q * a.rows, ms.tmp), ranges = min(a.ranges, total);
  if (u >= ranges) return;
  Walk w;
  w.at = range_begin(total, ranges, u);
  w.stop = range_begin(total, ranges, u + 1);
  w.item = attn_item_of(a, w.at, ms.tmp, &w.first);
  const int my_begin = w.at;

  if (threadIdx.x == 0) {
    ms.abort_flag = 0;
    for (int s = 0; s < kStages; ++s)
      for (int p = 0; p < kParts; ++p) {
        mbar_init(bar(B.full[s][p]), kProducers);
        mbar_init(bar(B.empty[s][p]), 1);
      }
    for (int i = 0; i < kInfo; ++i) mbar_init(bar(B.info[i]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B.sfull[i]), 1);
      mbar_init(bar(B.sfree[i]), 4);
      mbar_init(bar(B.done[i]), 1);
    }
    mbar_init(bar(B.pfull), 4);
    mbar_init(bar(B.pempty), 1);
    mbar_init(bar(B.qfull), kQThreads);
    mbar_init(bar(B.qempty), 1);
    mbar_init(bar(B.oempty), 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&ms.tmem), kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ms.tmem;

  if (warp >= 4 && warp < kMmaWarp) {
    // ======================= producers =======================
    // Each warp looks up all 64 tokens (lane l: 2 l, 2 l + 1), so that all
    // agree on which tiles are passed over; it copies tokens 4 pw + l / 8 + 16 j,
    // piece l % 8 of each 128-byte line.
    const LatentCache& C = a.cache;
    const int pw = warp - 4;
    struct Look {      // one unit of the stream
      int q, end, flags;
      int slot[2];     // entries (list) or slots
      int page[2];
    };
    // stage 1: the unit's entries
    auto entries = [&](Look& x, bool& more) {
      if (!more) {
        x.q = -1;
        return;
      }
      const int k = w.at - w.first;
      x.q = w.q;
      x.end = w.end;
      x.flags = (k == w.t1 - 1 ? 2 : 0) | (w.at + 1 == w.stop ? 4 : 0);
      const int e0 = k * kTok + 2 * lane;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.slot[i] = -1;
        if (a.list) {
          if (e0 + i < a.topk) x.slot[i] = __ldg(a.list + (int64_t)w.item * a.topk + e0 + i);
        } else {
          x.slot[i] = e0 + i;
        }
      }
      if (++w.at == w.first + w.t1) {
        more = w.at < w.stop;
        if (more) {
          w.first += w.n;
          ++w.item;
          w.open(a);
        }
      }
    };
    // stage 2: their pages
    auto pages = [&](Look& x) {
      if (x.q < 0) return;
      const int32_t* bt = C.bt + (int64_t)x.q * C.bt_stride;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (x.slot[i] >= x.end) x.slot[i] = -1;
        x.page[i] = x.slot[i] >= 0 ? __ldg(bt + (x.slot[i] >> C.log2b)) : 0;
      }
    };
    bool more = true;
    w.open(a);
    Look x0, x1, x2;
    entries(x0, more);
    entries(x1, more);
    pages(x0);
    int tile = 0;
    bool ok = true, fresh = true;
    const char* base = reinterpret_cast<const char*>(C.data) + (lane & 7) * 16;
    while (x0.q >= 0) {
      entries(x2, more);
      pages(x1);
      // rows and mask of x0
      int row[2];
      bool live[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        live[i] = x0.slot[i] >= 0;
        if (live[i] && (x0.page[i] < 0 || x0.page[i] >= C.num_pages)) {
          if (pw == 0) raise_error(a.err, ERR_PAGE, x0.q, (uint32_t)x0.page[i]);
          live[i] = false;
        }
        row[i] = live[i] ? (x0.page[i] << C.log2b) + (x0.slot[i] & (C.b - 1)) : -1;
      }
      const uint32_t even = __ballot_sync(0xffffffffu, live[0]), odd = __ballot_sync(0xffffffffu, live[1]);
      if (even || odd || (x0.flags & 2)) {  // a tile of which nothing is attended to is passed over
        const int st = tile % kStages;
        const uint32_t par = (uint32_t)(tile / kStages) & 1u;
        const char* src[4];
        uint32_t dst[4], bytes[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * pw + (lane >> 3) + 16 * j;
          const int r0 = __shfl_sync(0xffffffffu, row[0], t >> 1), r1 = __shfl_sync(0xffffffffu, row[1], t >> 1);
          const int r = (t & 1) ? r1 : r0;
          bytes[j] = r >= 0 ? 16u : 0u;  // 0: filled with zeros, nothing is read
          src[j] = base + (int64_t)(r >= 0 ? r : 0) * (kW * 2);
          dst[j] = kv_at + st * kStageBytes + t * 128 + (((lane & 7) ^ (t & 7)) << 4);
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
          const int p = j == 0 ? 4 : j - 1;  // kr first: S starts with it
          ok = wait_warp(bar(B.empty[st][p]), par ^ 1u, ctl);
          if (!ok) break;
          if (j == 0 && pw == 0 && lane == 0) {
            // the second product of tile - 4, the slot's last user, is done: tile - 2 took its stage
            Info& f = ms.info[tile % kInfo];
            f.even = even;
            f.odd = odd;
            f.flags = x0.flags | (fresh ? 1 : 0);
            mbar_arrive(bar(B.info[tile % kInfo]));
          }
#pragma unroll
          for (int b = 0; b < (p == 4 ? 1 : 2); ++b) {
            const int blk = p == 4 ? 8 : 2 * p + b;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst[i] + blk * kBlk),
                           "l"(src[i] + blk * 128), "r"(bytes[i])
                           : "memory");
          }
          // arrives when this thread's copies so far have landed
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(B.full[st][p])) : "memory");
        }
        if (!ok) break;
        fresh = x0.flags & 2;
        ++tile;
      }
      x0 = x1;
      x1 = x2;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kMmaWarp) {
    // ======================= first product =======================
    // The whole warp runs the loop; the elected lane issues.  The two
    // products are issued by two warps, each waiting for its own operands:
    // one warp that polled for both spent more time polling than the MMAs take.
    const uint32_t id_s = idesc_bf16(64, kTok, 0, 0);
    const uint64_t a2 = (uint64_t)(NH * 128 >> 4), b2 = kBlk >> 4;
    int seg = 0, flags = 0;
    bool ok = true;
    for (int tile = 0; ok && !(flags & 4); ++tile) {
      const int st = tile % kStages;
      ok = wait_warp(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, ctl);
      if (!ok) break;
      flags = __shfl_sync(0xffffffffu, ms.info[tile % kInfo].flags, 0);
      if (flags & 1) ok = wait_warp(bar(B.qfull), (uint32_t)seg & 1u, ctl);
      // S's buffer is that of two tiles ago
      if (ok && tile >= 2) ok = wait_warp(bar(B.sfree[tile & 1]), (uint32_t)((tile >> 1) - 1) & 1u, ctl);
      const uint32_t d = tmem + kSCol + (uint32_t)(tile & 1) * kTok;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        const int p = j == 0 ? 4 : j - 1;
        ok = ok && wait_warp(bar(B.full[st][p]), (uint32_t)(tile / kStages) & 1u, ctl);
        if (!ok) break;
        fence_async_smem();  // the copies are generic-proxy writes, the MMAs read through the async proxy
        fence_after();
        const uint64_t ad = sw128_desc(q_at + 2 * p * NH * 128, 16, 1024);
        const uint64_t bd = sw128_desc(kv_at + st * kStageBytes + 2 * p * kBlk, 16, 1024);
        if (elect()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f16(d, ad + 2 * kk, bd + 2 * kk, id_s, j > 0 || kk > 0 ? 1u : 0u);
          if (p == 4) {
            commit(bar(B.empty[st][4]));
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f16(d, ad + a2 + 2 * kk, bd + b2 + 2 * kk, id_s, 1u);
          }
          if (j == kParts - 1) {
            commit(bar(B.sfull[tile & 1]));
            if (flags & 2) commit(bar(B.qempty));
          }
        }
        __syncwarp();
      }
      if (flags & 2) ++seg;
    }
    // every MMA is complete before TMEM is given back
    if (elect()) commit(bar(B.done[0]));
    __syncwarp();
    drain(bar(B.done[0]), 0);
  } else if (warp == kMmaWarp + 1) {
    // ======================= second product =======================
    const uint32_t id_o = idesc_bf16(128, NH, 1, 0);
    int seg = 0, flags = 0;
    for (int tile = 0; !(flags & 4); ++tile) {
      const int st = tile % kStages;
      if (!wait_warp(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, ctl)) break;
      flags = __shfl_sync(0xffffffffu, ms.info[tile % kInfo].flags, 0);
      if (!wait_warp(bar(B.pfull), (uint32_t)tile & 1u, ctl)) break;
      if ((flags & 1) && seg > 0 && !wait_warp(bar(B.oempty), (uint32_t)(seg - 1) & 1u, ctl)) break;
      fence_after();
      const uint64_t ad = sw128_desc(kv_at + st * kStageBytes, kBlk, 1024), bd = sw128_desc(p_at, 16, 1024);
      const uint32_t joined = !(flags & 1);
      if (elect()) {
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk)
            mma_f16(tmem + mb * NH, ad + mb * (2 * kBlk >> 4) + kk * (2048 >> 4), bd + kk * 2, id_o,
                    kk > 0 ? 1u : joined);
          commit(bar(B.empty[st][mb]));
        }
        commit(bar(B.pempty));
      }
      __syncwarp();
      if (flags & 2) ++seg;
    }
    if (elect()) commit(bar(B.done[1]));
    __syncwarp();
    drain(bar(B.done[1]), 0);
  } else if (warp > kMmaWarp + 1) {
    // ======================= Q tiles =======================
    const int t = threadIdx.x - (kMmaWarp + 2) * 32;
    bool more = true;
    for (int seg = 0; more; ++seg) {
      w.open(a);
      if (seg > 0 && !wait_warp(bar(B.qempty), (uint32_t)(seg - 1) & 1u, ctl)) break;
      const char* ql = reinterpret_cast<const char*>(a.ql) + (int64_t)w.item * a.ql_tok * 2;
      const char* qr = reinterpret_cast<const char*>(a.qr) + (int64_t)w.item * a.qr_tok * 2;
      // 16-byte pieces: 72 a head, piece c of head h at block c / 8, row h, place (c % 8) ^ (h % 8)
      for (int i = t; i < NH * (kW / 8); i += kQThreads) {
        const int h = i / (kW / 8), c = i - h * (kW / 8);
        const uint32_t dst = q_at + (uint32_t)((c >> 3) * NH * 128 + h * 128 + (((c & 7) ^ (h & 7)) << 4));
        if (h0 + h < H) {
          const char* src = c < kDC / 8 ? ql + (int64_t)(h0 + h) * a.ql_head * 2 + c * 16
                                        : qr + (int64_t)(h0 + h) * a.qr_head * 2 + (c - kDC / 8) * 16;
          if (a.q_vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
          } else {  // queries that do not lie on 16 bytes
            const uint16_t* e = reinterpret_cast<const uint16_t*>(src);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = (uint32_t)e[2 * k] | (uint32_t)e[2 * k + 1] << 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                         "r"(v[3])
                         : "memory");
          }
        } else {
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      mbar_arrive(bar(B.qfull));
      more = w.next();
    }
  } else {
    // ======================= softmax and output =======================
    const int hA = 16 * warp + (lane >> 2);  // this thread's heads: hA, hA + 8
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t prow = p_at + (uint32_t)hA * 128 + (uint32_t)(lane & 3) * 4;
    const int sw = hA & 7;  // (hA + 8) & 7 is the same
    const bool mine = 16 * warp < NH;
    int tile = 0, seg = 0;
    bool run = true;
    while (run) {
      w.open(a);
      if (w.end == 0 && w.t0 == 0 && threadIdx.x == 0) raise_error(a.err, ERR_CTX_LEN, w.q, (uint32_t)a.ctx_len[w.q]);
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      int flags;
      bool alive = true;
      do {
        // ---- scores of the tile ----
        bool ok = wait_warp(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, ctl);
        ok = ok && wait_warp(bar(B.sfull[tile & 1]), (uint32_t)(tile >> 1) & 1u, ctl);
        uint32_t s[32];
        uint32_t even = 0, odd = 0;
        flags = 0;
        float t0 = -INFINITY, t1 = -INFINITY;
        if (ok) {
          even = ms.info[tile % kInfo].even;
          odd = ms.info[tile % kInfo].odd;
          flags = ms.info[tile % kInfo].flags;
        }
        if (ok && mine) {
          fence_after();
          tmem_ld_16x256b_x8(tmem + lanes + kSCol + (uint32_t)(tile & 1) * kTok, s);
          tmem_wait_ld();
          fence_before();
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(B.sfree[tile & 1]));
        if (ok && mine) {
          if ((even & odd) != 0xffffffffu) {
            // columns 8 n + 2 (lane % 4) and the next: bit 4 n + lane % 4 of the two
            const uint32_t ev = even >> (lane & 3), od = odd >> (lane & 3);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              if (!(ev >> (4 * n) & 1)) s[4 * n] = s[4 * n + 2] = 0xff800000u;
              if (!(od >> (4 * n) & 1)) s[4 * n + 1] = s[4 * n + 3] = 0xff800000u;
            }
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            t0 = fmaxf(t0, fmaxf(__uint_as_float(s[4 * n]), __uint_as_float(s[4 * n + 1])));
            t1 = fmaxf(t1, fmaxf(__uint_as_float(s[4 * n + 2]), __uint_as_float(s[4 * n + 3])));
          }
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
          t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2)) * a.scale_log2;
          t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2)) * a.scale_log2;
        }
        // ---- the reference moves where a row outgrew it ----
        const bool grow = mine && (t0 > m0 + kLazy || t1 > m1 + kLazy);
        if (bar_or(1, 128, grow || !ok)) {
          // (the second product of the tile before has read the weights and O is whole)
          if (ok && tile > 0) ok = wait_warp(bar(B.pempty), (uint32_t)(tile - 1) & 1u, ctl);
          if (mine) {
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            const float f0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
            l0 *= f0;
            l1 *= f1;
            m0 = n0;
            m1 = n1;
            if ((lane & 3) == 0) {
              ms.fac[hA] = f0;
              ms.fac[hA + 8] = f1;
            }
          }
          if (bar_or(1, 128, !ok)) {
            alive = false;
            break;
          }
          if (!(flags & 1)) {
            fence_after();
#pragma unroll 1
            for (int c = 0; c < 4 * NH; c += 16) {
              uint32_t o[16];
              tmem_ld16(tmem + lanes + (uint32_t)c, o);
              tmem_wait_ld();
              const float4* f4 = reinterpret_cast<const float4*>(ms.fac + c % NH);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = f4[i];
                o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * f.x);
                o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * f.y);
                o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * f.z);
                o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * f.w);
              }
              tmem_st16(tmem + lanes + (uint32_t)c, o);
            }
            tmem_wait_st();
          }
          bar_sync(1, 128);  // the factors have been read
        }
        // ---- weights ----
        if (mine) {
          const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float p0 = ex2(fmaf(__uint_as_float(s[4 * n]), a.scale_log2, -r0));
            const float p1 = ex2(fmaf(__uint_as_float(s[4 * n + 1]), a.scale_log2, -r0));
            const float p2 = ex2(fmaf(__uint_as_float(s[4 * n + 2]), a.scale_log2, -r1));
            const float p3 = ex2(fmaf(__uint_as_float(s[4 * n + 3]), a.scale_log2, -r1));
            l0 += p0 + p1;
            l1 += p2 + p3;
            s[2 * n] = pack_bf16(p0, p1);
            s[2 * n + 1] = pack_bf16(p2, p3);
          }
        }
        ok = tile == 0 || wait_warp(bar(B.pempty), (uint32_t)(tile - 1) & 1u, ctl);
        if (ok && mine) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const uint32_t at = prow + (uint32_t)((n ^ sw) << 4);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(s[2 * n]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(s[2 * n + 1]) : "memory");
          }
          fence_async_smem();
        }
        // a wait that ran out here is met again at the next tile's barrier or the item's end
        fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(B.pfull));
        ++tile;
      } while (!(flags & 2));
      if (!alive) break;

      // ---- the item's end ----
      bool ok = wait_warp(bar(B.pempty), (uint32_t)(tile - 1) & 1u, ctl);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      const int64_t part = (int64_t)blockIdx.x * 2 + (w.first <= my_begin ? 0 : 1);
      if (mine && (lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = hA + 8 * i;
          const float m = i ? m1 : m0, l = i ? l1 : l0;
          if (whole) {
            ms.fac[h] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (a.lse && h0 + h < H)
              a.lse[(int64_t)w.item * H + h0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
          } else {
            a.part_ml[part * NH + h] = make_float2(m, l);
          }
        }
      }
      if (bar_or(1, 128, !ok)) break;
      fence_after();
      const int nh = min(NH, H - h0);
#pragma unroll 1
      for (int mb = 0; mb < 4; ++mb) {
        const int d = mb * 128 + warp * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < NH; c += 16) {
          uint32_t o[16];
          tmem_ld16(tmem + lanes + (uint32_t)(mb * NH + c), o);
          tmem_wait_ld();
          if (whole) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) +
                                 ((int64_t)w.item * H + h0 + c + (lane & 1)) * kDC + (d & ~1);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              // neighbouring lanes trade halves: each gets two columns of one head
              const float x = __uint_as_float(o[i]) * ms.fac[c + i], y = __uint_as_float(o[i + 1]) * ms.fac[c + i + 1];
              const float z = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x : y, 1);
              if (c + i + (lane & 1) < nh)
                *reinterpret_cast<uint32_t*>(out + (int64_t)i * kDC) = (lane & 1) ? pack_bf16(z, y) : pack_bf16(x, z);
            }
          } else {
            float* out = a.part + (part * NH + c) * kDC + d;
#pragma unroll
            for (int i = 0; i < 16; ++i) out[(int64_t)i * kDC] = __uint_as_float(o[i]);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B.oempty));
      bar_sync(1, 128);  // the factors have been read
      ++seg;
      run = w.next();
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool attn_tc_supported(const AttnArgs& a, int bf16) {
  // cache rows are 32-bit numbers
  return bf16 && a.cache.dc == kDC && a.cache.dr == kDR && ((uintptr_t)a.cache.data & 15) == 0 &&
         ((int64_t)a.cache.num_pages << a.cache.log2b) < (int64_t(1) << 31) && ((uintptr_t)a.out & 3) == 0;
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) {
  const uint32_t smem = smem_bytes(a.group);
  cudaError_t e = cudaFuncSetAttribute(k_attn_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch l(dim3((unsigned)(a.ranges * a.ngroups)), dim3(kThreads), smem, s);
  return cudaLaunchKernelEx(&l.cfg, k_attn_tc, a);
}

}  // namespace spin
