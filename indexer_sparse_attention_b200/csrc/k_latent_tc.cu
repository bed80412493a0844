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
// Warps (480 threads, one block per SM):
//   0..7  softmax: S from TMEM (warp w: heads 16 (w % 4) .. + 15, tokens
//         32 (w / 4) .. + 31), weights to shared memory; at an item's end O^T
//         from TMEM to the output or to the block's share
//   8..11 producers: 16-byte asynchronous copies, eight lanes a 128-byte line.  A
//         gather by TMA (four rows a request) moved 2.0 TB/s from one warp's
//         lanes and 4.3 TB/s from four warps, these copies 6.45 TB/s (64 rows of
//         1152 bytes at random from 302 MB, 148 blocks).  An item's queries
//         come the same way, as a tile whose rows are its heads
//   12, 13  issue of the first and of the second product
//   14    look-up, up to four tiles ahead: list entries -> pages -> cache rows,
//         which it also asks into L2 (a tile's copies then take 1580 cycles under
//         load, not 2450 to 3350)
// Two 72 KB token tiles in flight, each cut into five parts (the rotary part
// and four of 128 latent columns) with their own barriers: a part is
// reloaded as soon as the second product has read its columns, and S starts
// on the parts that have landed.
//
// Whole calls, the join included: 97 us for 96 requests x 128 heads x 2048 listed
// slots (560 TFLOP/s, 2.6 TB/s).  There a tile takes 2960 cycles.  Its products
// read both operands from shared memory, 144 KB for S and 96 KB for the second, and 72 KB
// come in: 2440 cycles at 128 bytes each; the rest is the chain copy, S, softmax,
// second product of the two tiles that fit beside 72 KB of queries.  61 us for 32
// requests x 4 rows x 16 heads x 2048 slots, 5.0 TB/s, in steady state at HBM's
// rate, then the start (7 us of dependent reads: length, list, page, entry) and
// the outputs.  The CUDA-core kernel takes 14.5 ms for the first.
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
constexpr int kThreads = 480;
constexpr int kSoft = 256, kProducers = 128;  // threads of the softmax and of the copies
constexpr int kCopyWarp = 8, kMmaWarp = 12, kLookWarp = 14;
constexpr float kLazy = 8.0f;
constexpr uint32_t kSCol = 256;                  // S buffers behind O^T's 4 * 64 columns
constexpr uint32_t kTmemCols = 512;

struct Info {
  uint32_t even, odd;  // the even and the odd tokens that are attended to
  int flags;           // 1: first tile of an item's share, 2: its last, 4: the block's last
  int item;
  int row[kTok];       // cache rows, -1: not attended to
};

struct Bars {
  uint64_t full[kStages][kParts];   // copies landed
  uint64_t empty[kStages][kParts];  // MMAs that read the part
  uint64_t info[kInfo];             // tile info written
  uint64_t infofree[kInfo];         // and no longer needed: the tile's second product is complete
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
  uint32_t tmem;
  int abort_flag;
};

constexpr int kPBytes = kTcHeads * 128;  // the weights, at an item's end a place to transpose its output
__host__ __device__ constexpr uint32_t smem_bytes(int nh) {
  return 1024 + (uint32_t)(kBlocks * nh * 128 + kStages * kStageBytes + kPBytes) + (uint32_t)sizeof(Misc);
}
static_assert(smem_bytes(kTcHeads) <= 227 * 1024, "one block's shared memory");

// The walk over a block's items: `whole` of them whole, then its units [at,
// stop) of the others, of which the current item starts at unit `first`.
struct Walk {
  int item, whole, later;  // later: the first item that is not whole
  int first, at, stop;
  int q, r, n, t0, t1;
  __device__ __forceinline__ void open(const AttnArgs& a) {
    q = item / a.rows;
    r = item - q * a.rows;
    n = attn_tiles(a, a.list ? 0 : attn_end(a, q, r));  // (lists: the length is not waited for)
    t0 = whole > 0 ? 0 : at - first;
    t1 = whole > 0 ? n : min(n, stop - first);
  }
  __device__ __forceinline__ bool last() const { return whole > 0 ? whole == 1 && at >= stop : first + t1 >= stop; }
  __device__ __forceinline__ bool next() {  // false: nothing left
    if (last()) return false;
    if (whole > 0) {
      item = --whole ? item + 1 : later;
    } else {
      at = first + t1;
      first += n;
      ++item;
    }
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tc(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NH = a.group, H = a.H;
  // Q first: the M = 64 rows of S's A operand run past the NH rows of a
  // block of Q into what follows (rows that nothing reads)
  uint8_t* q_sm = smem;
  uint8_t* kv_sm = q_sm + kBlocks * NH * 128;
  uint8_t* p_sm = kv_sm + kStages * kStageBytes;
  Misc& ms = *reinterpret_cast<Misc*>(p_sm + kPBytes);
  const uint32_t q_at = smem_u32(q_sm), kv_at = smem_u32(kv_sm), p_at = smem_u32(p_sm);
  Bars& B = ms.bars;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const Ctl ctl{&ms.abort_flag, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x % a.ngroups, u = blockIdx.x / a.ngroups;
  const int h0 = g * NH;

  // what does not depend on the kernel before runs while that ends
  if (threadIdx.x == 0) {
    ms.abort_flag = 0;
    for (int s = 0; s < kStages; ++s)
      for (int p = 0; p < kParts; ++p) {
        mbar_init(bar(B.full[s][p]), kProducers);
        mbar_init(bar(B.empty[s][p]), 1);
      }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(bar(B.info[i]), 1);
      mbar_init(bar(B.infofree[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B.sfull[i]), 1);
      mbar_init(bar(B.sfree[i]), kSoft / 32);
      mbar_init(bar(B.done[i]), 1);
    }
    mbar_init(bar(B.pfull), kSoft / 32);
    mbar_init(bar(B.pempty), 1);
    mbar_init(bar(B.qfull), kProducers);
    mbar_init(bar(B.qempty), 1);
    mbar_init(bar(B.oempty), kSoft / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // TMEM is taken behind the wait and held before the release: a kernel that
  // still waits for the one before never holds columns which that may need, and
  // its own successor is not there yet.
  pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&ms.tmem), kTmemCols);

  // the block's items and units (all threads)
  Walk w;
  {
    const Place at = attn_place(a, -1, u, reinterpret_cast<int*>(ms.info));
    w.whole = a.whole;
    w.later = at.item;
    w.first = at.first;
    w.at = w.stop = 0;
    if (u < at.ranges) {
      w.at = range_begin(at.total, at.ranges, u);
      w.stop = range_begin(at.total, at.ranges, u + 1);
    }
    w.item = w.whole ? u * w.whole : w.later;
    fence_before();
    __syncthreads();
    fence_after();
  }
  const uint32_t tmem = ms.tmem;
  pdl_release();
  const int my_begin = w.at;
  const bool any = w.whole || w.at < w.stop;

  if (!any) {
    // more blocks than units
  } else if (warp == kLookWarp) {
    // ======================= look-up =======================
    // Lane l takes tokens 2 l and 2 l + 1, two units at a time.
    const LatentCache& C = a.cache;
    const char* data = reinterpret_cast<const char*>(C.data);
    struct Look {
      int item, q, r, ctx, flags;
      int slot[2], page[2];
    };
    int tile = 0;
    bool more = true, ok = true, fresh = true;
    w.open(a);
    int k = w.t0;
    while (more && ok) {
      Look x[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {  // the list's entries
        x[v].q = -1;
        if (!more) continue;
        x[v].item = w.item;
        x[v].q = w.q;
        x[v].r = w.r;
        x[v].ctx = __ldg(a.ctx_len + w.q);
        x[v].flags = k < w.t1 - 1 ? 0 : w.last() ? 6 : 2;
        const int e0 = k * kTok + 2 * lane;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[v].slot[i] = -1;
          if (a.list) {
            if (e0 + i < a.topk) x[v].slot[i] = __ldg(a.list + (int64_t)w.item * a.topk + e0 + i);
          } else {
            x[v].slot[i] = e0 + i;
          }
        }
        if (++k == w.t1) {
          more = w.next();
          if (more) {
            w.open(a);
            k = w.t0;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < 2; ++v)  // their pages
        if (x[v].q >= 0) {
          const int32_t* bt = C.bt + (int64_t)x[v].q * C.bt_stride;
          const int end = attn_end_at(a, x[v].ctx, x[v].r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (x[v].slot[i] >= end) x[v].slot[i] = -1;
            x[v].page[i] = x[v].slot[i] >= 0 ? __ldg(bt + (x[v].slot[i] >> C.log2b)) : 0;
          }
        }
#pragma unroll
      for (int v = 0; v < 2; ++v) {  // cache rows and mask
        if (x[v].q < 0 || !ok) continue;
        int row[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bool live = x[v].slot[i] >= 0;
          if (live && (x[v].page[i] < 0 || x[v].page[i] >= C.num_pages)) {
            raise_error(a.err, ERR_PAGE, x[v].q, (uint32_t)x[v].page[i]);
            live = false;
          }
          row[i] = live ? (x[v].page[i] << C.log2b) + (x[v].slot[i] & (C.b - 1)) : -1;
          if (live) {
#pragma unroll
            for (int c = 0; c < kBlocks; ++c)  // (one bulk prefetch a row instead took 40 cycles a row to issue)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(data + (int64_t)row[i] * (kW * 2) + c * 128) : "memory");
          }
        }
        const uint32_t even = __ballot_sync(0xffffffffu, row[0] >= 0), odd = __ballot_sync(0xffffffffu, row[1] >= 0);
        if (!even && !odd && !(x[v].flags & 2)) continue;  // nothing of the tile is attended to
        const int at = tile % kInfo;
        if (tile >= kInfo) ok = wait_warp(bar(B.infofree[at]), (uint32_t)(tile / kInfo - 1) & 1u, ctl);
        if (!ok) continue;
        Info& f = ms.info[at];
        f.row[2 * lane] = row[0];
        f.row[2 * lane + 1] = row[1];
        if (lane == 0) {
          f.even = even;
          f.odd = odd;
          f.flags = x[v].flags | (fresh ? 1 : 0);
          f.item = x[v].item;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B.info[at]));
        fresh = x[v].flags & 2;
        ++tile;
      }
    }
  } else if (warp >= kCopyWarp && warp < kMmaWarp) {
    // ======================= producers =======================
    // This thread copies piece lane % 8 of each 128-byte line of tokens row0 + 16 j.
    const int pw = warp - kCopyWarp;
    const char* data = reinterpret_cast<const char*>(a.cache.data);
    // this thread's 4 rows' copies of one 64-column block
    const int piece = lane & 7, row0 = 4 * pw + (lane >> 3);
    auto copy = [&](uint32_t dst, const char* src, uint32_t bytes) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    };
    // arrives when this thread's copies so far have landed
    auto landed = [&](uint64_t& b) {
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(b)) : "memory");
    };
    auto queries = [&](int item) {
      const char* ql = reinterpret_cast<const char*>(a.ql) + (int64_t)item * a.ql_tok * 2;
      const char* qr = reinterpret_cast<const char*>(a.qr) + (int64_t)item * a.qr_tok * 2;
#pragma unroll 1
      for (int h = row0; h < NH; h += 16) {
        const bool live = h0 + h < H;  // else zeros
        const char* l = ql + (int64_t)(live ? h0 + h : 0) * a.ql_head * 2 + piece * 16;
        const char* r = qr + (int64_t)(live ? h0 + h : 0) * a.qr_head * 2 + piece * 16;
        const uint32_t dst = q_at + h * 128 + ((piece ^ (h & 7)) << 4);
        if (a.q_vec) {
#pragma unroll
          for (int blk = 0; blk < kBlocks; ++blk) copy(dst + blk * NH * 128, blk < 8 ? l + blk * 128 : r, live ? 16u : 0u);
        } else {  // queries that do not lie on 16 bytes
#pragma unroll 1
          for (int blk = 0; blk < kBlocks; ++blk) {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(blk < 8 ? l + blk * 128 : r);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = live ? (uint32_t)e[2 * k] | (uint32_t)e[2 * k + 1] << 16 : 0u;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + blk * NH * 128), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3])
                         : "memory");
          }
        }
      }
      if (a.q_vec) {
        landed(B.qfull);
      } else {  // plain stores: no asynchronous arrival stands for them, and the product reads through the async proxy
        fence_async_smem();
        mbar_arrive(bar(B.qfull));
      }
    };
    queries(w.item);
    int seg = 0, flags = 0;
    for (int tile = 0; !(flags & 4); ++tile) {
      const int st = tile % kStages;
      const uint32_t par = (uint32_t)(tile / kStages) & 1u ^ 1u;
      if (!wait_warp2(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, bar(B.empty[st][4]), par, ctl)) break;
      const Info& f = ms.info[tile % kInfo];
      flags = f.flags;
      const int item = f.item;
      const char* src[4];
      uint32_t dst[4], bytes[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = row0 + 16 * j, r = f.row[t];
        bytes[j] = r >= 0 ? 16u : 0u;  // 0: filled with zeros, nothing is read
        src[j] = data + piece * 16 + (int64_t)(r >= 0 ? r : 0) * (kW * 2);
        dst[j] = kv_at + st * kStageBytes + t * 128 + ((piece ^ (t & 7)) << 4);
      }
      auto block = [&](int blk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy(dst[i] + blk * kBlk, src[i] + blk * 128, bytes[i]);
      };
      block(8);  // kr first: S starts with it
      landed(B.full[st][4]);
      bool ok = true;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        ok = ok && wait_warp(bar(B.empty[st][p]), par, ctl);
        if (!ok) break;
        block(2 * p);
        block(2 * p + 1);
        landed(B.full[st][p]);
      }
      if (!ok) break;
      if ((flags & 1) && seg > 0) {
        // (behind the tile's copies: those wait for the second product of two tiles ago, the queries' place for
        // the first product of the last, which comes later)
        if (!wait_warp(bar(B.qempty), (uint32_t)(seg - 1) & 1u, ctl)) break;
        queries(item);
      }
      if (flags & 2) ++seg;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kMmaWarp) {
    // ======================= first product =======================
    // The whole warp runs the loop; the elected lane issues.  The two
    // products are issued by two warps, each waiting for its own operands:
    // one warp that polled for both spent more time polling than the MMAs take.
    const uint32_t id_s = idesc_bf16(64, kTok, 0, 0);
    const uint64_t a1 = (uint64_t)(NH * 128 >> 4), b1 = kBlk >> 4;  // a 64-column block further
    int seg = 0, flags = 0;
    for (int tile = 0; !(flags & 4); ++tile) {
      const int st = tile % kStages;
      const uint32_t par = (uint32_t)(tile / kStages) & 1u;
      // S's buffer is that of two tiles ago (an untouched barrier has "completed" parity 1)
      if (!wait_warp2(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, bar(B.sfree[tile & 1]),
                      (uint32_t)(tile >> 1) & 1u ^ 1u, ctl))
        break;
      flags = __shfl_sync(0xffffffffu, ms.info[tile % kInfo].flags, 0);
      if ((flags & 1) && !wait_warp(bar(B.qfull), (uint32_t)seg & 1u, ctl)) break;
      const uint32_t d = tmem + kSCol + (uint32_t)(tile & 1) * kTok;
      const uint64_t ad = sw128_desc(q_at, 16, 1024), bd = sw128_desc(kv_at + st * kStageBytes, 16, 1024);
      auto block = [&](int blk) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16(d, ad + blk * a1 + 2 * kk, bd + blk * b1 + 2 * kk, id_s, blk < 8 || kk > 0 ? 1u : 0u);
      };
      // kr and the first half of c, then the second half
      if (!wait_warp2(bar(B.full[st][4]), par, bar(B.full[st][1]), par, ctl)) break;  // (part 0 lands before part 1)
      fence_async_smem();  // the copies are generic-proxy writes, the MMAs read through the async proxy
      fence_after();
      if (elect()) {
        block(8);
        commit(bar(B.empty[st][4]));
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) block(blk);
      }
      __syncwarp();
      if (!wait_warp2(bar(B.full[st][2]), par, bar(B.full[st][3]), par, ctl)) break;
      fence_async_smem();
      if (elect()) {
#pragma unroll
        for (int blk = 4; blk < 8; ++blk) block(blk);
        commit(bar(B.sfull[tile & 1]));
        if (flags & 2) commit(bar(B.qempty));
      }
      __syncwarp();
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
      if (!wait_warp2(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, bar(B.pfull), (uint32_t)tile & 1u, ctl))
        break;
      flags = __shfl_sync(0xffffffffu, ms.info[tile % kInfo].flags, 0);
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
        commit(bar(B.infofree[tile % kInfo]));
      }
      __syncwarp();
      if (flags & 2) ++seg;
    }
    if (elect()) commit(bar(B.done[1]));
    __syncwarp();
    drain(bar(B.done[1]), 0);
  } else {
    // ======================= softmax and output =======================
    const int quarter = warp & 3, half = warp >> 2;
    const int hA = 16 * quarter + (lane >> 2);  // this thread's heads: hA, hA + 8
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_at = tmem + lanes + kSCol + (uint32_t)half * 32;
    const uint32_t prow = p_at + (uint32_t)hA * 128 + (uint32_t)(lane & 3) * 4;
    const int sw = hA & 7;  // (hA + 8) & 7 is the same
    const bool mine = 16 * quarter < NH;
    // the two token halves' maxima, then sums, where the weights lie (while no product reads those)
    float(*halves)[kTcHeads] = reinterpret_cast<float(*)[kTcHeads]>(p_sm);
    int tile = 0;
    bool run = true;
    while (run) {
      w.open(a);
      if (threadIdx.x == 0 && w.t0 == 0 && attn_end(a, w.q, w.r) == 0)
        raise_error(a.err, ERR_CTX_LEN, w.q, (uint32_t)a.ctx_len[w.q]);
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // references (scores) and sums
      float r0 = 0.f, r1 = 0.f, far0 = 0.f, far1 = 0.f;  // references times the factor, or (far ones) as they are
      int flags;
      bool alive = true;
      do {
        // ---- scores of the tile ----
        // (S of the tile, and the weights' place: the second product of the tile before has read it, and O is whole)
        bool ok = wait_warp3(bar(B.info[tile % kInfo]), (uint32_t)(tile / kInfo) & 1u, bar(B.sfull[tile & 1]),
                             (uint32_t)(tile >> 1) & 1u, bar(B.pempty), (uint32_t)tile & 1u ^ 1u, ctl);
        uint32_t s[16], p[8];
        flags = 0;
        if (ok) {
          flags = ms.info[tile % kInfo].flags;
          const uint32_t even = ms.info[tile % kInfo].even, odd = ms.info[tile % kInfo].odd;
          if (mine) {
            fence_after();
            tmem_ld_16x256b_x4(s_at + (uint32_t)(tile & 1) * kTok, s);
            tmem_wait_ld();
            fence_before();
            if ((even & odd) != 0xffffffffu) {
              // columns 32 half + 8 n + 2 (lane % 4) and the next: bit 16 half + 4 n + lane % 4 of the two
              const uint32_t ev = even >> (16 * half + (lane & 3)), od = odd >> (16 * half + (lane & 3));
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                if (!(ev >> (4 * n) & 1)) s[4 * n] = s[4 * n + 2] = 0xff800000u;
                if (!(od >> (4 * n) & 1)) s[4 * n + 1] = s[4 * n + 3] = 0xff800000u;
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B.sfree[tile & 1]));
        }
        // ---- weights by the reference that there is; where a row outgrew it, it moves and they are taken again ----
        float d0, d1;
        for (int pass = 0;; ++pass) {
          bool grow = flags & 1;  // (the first tile: there is no reference yet)
          d0 = d1 = 0.f;
          if (ok && mine && (pass || !(flags & 1))) {
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              float x[4];  // two tokens of each head: (score - far) * scale - r
              sub2(x[0], x[1], __uint_as_float(s[4 * n]), __uint_as_float(s[4 * n + 1]), far0);
              sub2(x[2], x[3], __uint_as_float(s[4 * n + 2]), __uint_as_float(s[4 * n + 3]), far1);
              fma2(x[0], x[1], x[0], x[1], a.scale_log2, -r0);
              fma2(x[2], x[3], x[2], x[3], a.scale_log2, -r1);
              x0 = fmaxf(x0, fmaxf(x[0], x[1]));
              x1 = fmaxf(x1, fmaxf(x[2], x[3]));
              const float p0 = ex2(x[0]), p1 = ex2(x[1]), p2 = ex2(x[2]), p3 = ex2(x[3]);
              d0 += p0 + p1;
              d1 += p2 + p3;
              p[2 * n] = pack_bf16(p0, p1);
              p[2 * n + 1] = pack_bf16(p2, p3);
            }
            grow = x0 > (m0 == -INFINITY ? -INFINITY : kLazy) || x1 > (m1 == -INFINITY ? -INFINITY : kLazy);
          }
          if (pass || !bar_or(1, kSoft, grow || !ok)) break;
          float t0 = -INFINITY, t1 = -INFINITY;
          if (ok && mine) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              t0 = fmaxf(t0, fmaxf(__uint_as_float(s[4 * n]), __uint_as_float(s[4 * n + 1])));
              t1 = fmaxf(t1, fmaxf(__uint_as_float(s[4 * n + 2]), __uint_as_float(s[4 * n + 3])));
            }
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
            }
            if ((lane & 3) == 0) {
              halves[half][hA] = t0;
              halves[half][hA + 8] = t1;
            }
          }
          alive = !bar_or(1, kSoft, !ok);
          if (!alive) break;
          if (mine) {
            const float n0 = fmaxf(m0, fmaxf(t0, halves[half ^ 1][hA]));
            const float n1 = fmaxf(m1, fmaxf(t1, halves[half ^ 1][hA + 8]));
            const float f0 = n0 == -INFINITY ? 1.f : moved(m0, n0, a.scale_log2);
            const float f1 = n1 == -INFINITY ? 1.f : moved(m1, n1, a.scale_log2);
            l0 *= f0;
            l1 *= f1;
            m0 = n0;
            m1 = n1;
            r0 = m0 == -INFINITY ? 0.f : m0 * a.scale_log2;
            r1 = m1 == -INFINITY ? 0.f : m1 * a.scale_log2;
            far0 = far1 = 0.f;
            if (fabsf(r0) >= kFar) {
              far0 = m0;
              r0 = 0.f;
            }
            if (fabsf(r1) >= kFar) {
              far1 = m1;
              r1 = 0.f;
            }
            if (half == 0 && (lane & 3) == 0) {
              ms.fac[hA] = f0;
              ms.fac[hA + 8] = f1;
            }
          }
          bar_sync(1, kSoft);  // the factors are there, the halves' maxima have been read
          if (!(flags & 1)) {
            fence_after();
#pragma unroll 1
            for (int c = 2 * half * NH; c < 2 * (half + 1) * NH; c += 16) {
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
            bar_sync(1, kSoft);  // the factors have been read
          }
        }
        if (!alive) break;
        l0 += d0;
        l1 += d1;
        if (mine) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t at = prow + (uint32_t)(((4 * half + n) ^ sw) << 4);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(p[2 * n]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(p[2 * n + 1]) : "memory");
          }
          fence_async_smem();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B.pfull));
        ++tile;
      } while (!(flags & 2));
      if (!alive) break;

      // ---- the item's end ----
      bool ok = wait_warp(bar(B.pempty), (uint32_t)(tile - 1) & 1u, ctl);
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
      }
      if (half == 1 && mine && (lane & 3) == 0) {
        halves[1][hA] = l0;
        halves[1][hA + 8] = l1;
      }
      if (bar_or(1, kSoft, !ok)) break;
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      const int64_t part = (int64_t)blockIdx.x * 2 + (w.first <= my_begin ? 0 : 1);
      if (half == 0 && mine && (lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = hA + 8 * i;
          const float m = (i ? m1 : m0) * a.scale_log2, l = (i ? l1 : l0) + halves[1][h];
          if (whole) {
            ms.fac[h] = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            if (a.lse && h0 + h < H)
              a.lse[(int64_t)w.item * H + h0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * (1.f / kLog2e);
          } else {
            a.part_ml[part * NH + h] = make_float2(m, l);
          }
        }
      }
      bar_sync(1, kSoft);
      fence_after();
      const int nh = min(NH, H - h0);
      // 16 heads x 128 columns at a time; the two halves take 256 columns each
      __nv_bfloat16* turn = reinterpret_cast<__nv_bfloat16*>(p_sm) + half * 16 * 128;  // [16 heads][128 columns]
      const int t128 = threadIdx.x & 127;
#pragma unroll 1
      for (int i = 0; i < 2 * NH; i += 16) {
        uint32_t o[16];
        tmem_ld16(tmem + lanes + (uint32_t)(2 * half * NH + i), o);
        const int mb = i >= NH, c = i - mb * NH, d = (2 * half + mb) * 128;
        tmem_wait_ld();
        if (whole) {
          // 16 bytes a thread, by way of the weights' place
          float4 f[4];  // (all read before the first store, which might alias them)
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = *reinterpret_cast<const float4*>(ms.fac + c + 4 * k);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            __nv_bfloat16* at = turn + 4 * k * 128 + quarter * 32 + lane;
            at[0] = __float2bfloat16_rn(__uint_as_float(o[4 * k]) * f[k].x);
            at[128] = __float2bfloat16_rn(__uint_as_float(o[4 * k + 1]) * f[k].y);
            at[256] = __float2bfloat16_rn(__uint_as_float(o[4 * k + 2]) * f[k].z);
            at[384] = __float2bfloat16_rn(__uint_as_float(o[4 * k + 3]) * f[k].w);
          }
          bar_sync(2 + half, 128);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = 8 * j + (t128 >> 4), col = (t128 & 15) * 8;
            if (c + k < nh)
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                        ((int64_t)w.item * H + h0 + c + k) * kDC + d + col) =
                  *reinterpret_cast<const uint4*>(turn + k * 128 + col);
          }
          bar_sync(2 + half, 128);
        } else {
          float* sh = a.part + (part * NH + c) * kDC + d + quarter * 32 + lane;
#pragma unroll
          for (int k = 0; k < 16; ++k) sh[k * kDC] = __uint_as_float(o[k]);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B.oempty));
      bar_sync(1, kSoft);  // the factors have been read
      run = w.next();
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

// bf16 at these widths and 16-byte alignment; all else takes the CUDA-core kernel.
bool attn_tc_supported(const AttnArgs& a, int bf16) {
  // cache rows are 32-bit numbers
  return bf16 && a.cache.dc == kDC && a.cache.dr == kDR && ((uintptr_t)a.cache.data & 15) == 0 &&
         ((int64_t)a.cache.num_pages << a.cache.log2b) < (int64_t(1) << 31) && ((uintptr_t)a.out & 15) == 0;
}

cudaError_t prepare_attn_tc() {
  return cudaFuncSetAttribute(k_attn_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kTcHeads));
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) {
  PdlLaunch l(dim3((unsigned)(a.ranges * a.ngroups)), dim3(kThreads), smem_bytes(a.group), s);
  return cudaLaunchKernelEx(&l.cfg, k_attn_tc, a);
}

}  // namespace spin
