// k_prefill_tc.cu -- expanded latent attention on the 5th-generation tensor
// cores: bf16, latent width 512, key width 128 + 64 (rotary), value width 128.
//
// k_expand_tc   [k | v] = W_h c for every slot and head, into the workspace: a
//               matrix product M = slots, N = 128 twice, K = 512.  A block keeps
//               the latents of 128 slots in TMEM and streams the heads' weights,
//               160 KB in flight, so L2 -> SM carries 256 KB a unit (slot tile,
//               head) instead of 384.  109 us for 16K slots x 32 heads, 1.26
//               PFLOP/s, where a large plain product reaches 1.65: a unit
//               takes some 4800 cycles, its products alone 4160, bringing in a
//               slot tile 6000.
// k_prefill_tc  causal attention of 256 rows of one head: two 128-row tiles take
//               turns on the tensor cores, one's softmax under the other's
//               products:
//   S_t [128 x 128 keys] = Q_t . K^T   M 128, N 128, K 192 (shared memory both)
//   O_t [128 x 128]     += P_t . V     M 128, N 128, K 128 (P from TMEM)
//               P (bf16) overwrites its S in TMEM.  A thread owns a row, so
//               maximum, sum and rescaling need no exchange; the softmax
//               reference moves only where a row's maximum has grown by more
//               than 8 (log2 units), and then its warp rescales O.  K and V come
//               in 16 KB blocks (K: 64 columns of the 128 keys, V: 64 keys)
//               through one ring of eight, in the order of use.  For 4096 rows
//               at the end of 16K slots x 32 heads some 945 us (1.27 PFLOP/s) of
//               the call's 1075, on a cool card; in a steady run the power limit
//               takes a tenth of the clock.  Bound by the products, which read 128 bytes of shared
//               memory a cycle in S (all there is), together with the chain S ->
//               weights -> second product -> S of each row tile: P takes the place
//               of its S, and TMEM has no room for another.  Without the softmax
//               the call took 0.98 ms instead of 1.09.
//
// Rounded to bf16, each at most half a step, 2^-8: the expanded keys and values,
// as a model that keeps them would round them, and the weights P for the second
// product.  The sums of the weights are of the unrounded ones, all sums fp32.  On
// some tens of tokens the 2-norm of the error is up to 0.0034 of the output's,
// 0.0017 of it from the output's own rounding, as much from V's; it falls with the
// context's length.  fp16 would take less (0.0024), but holds values of any
// magnitude only with a factor, which a row would share with slots that it does
// not see or hardly weighs: its own values and weights then fall below fp16's
// smallest where such a slot is some 2^14 times larger.
//
// The CUDA-core kernels of the same steps took 260 ms where these take 1.08.
#include <algorithm>

#include "latent_internal.cuh"
#include "umma.cuh"

namespace spin {
namespace {

using namespace umma;

constexpr int kDC = 512, kDR = 64, kDN = 128, kDV = 128, kN = kDN + kDV;
constexpr int kRowTile = 128;
constexpr int kBlk = kRowTile * 128;  // 128 rows of 64 columns
constexpr float kLazy = 8.0f;
constexpr int kNoSlot = 0x7fffffff;

// ---------------------------------------------------------------------------
// expansion
// ---------------------------------------------------------------------------
// warps 0..3 half of the latents' columns and the keys' epilogue, 4..7 the other half and the values', 8 copies, 9 MMA
// issue
constexpr int kExpThreads = 320;
constexpr int kHalf = kN / 2;        // a unit's product is taken in two halves, the keys and the values
constexpr int kStageK = 128;         // reduction width of a stage of weights
constexpr int kBBytes = kHalf * kStageK * 2;
constexpr int kBStages = 5;
constexpr int kOutBufs = 2;          // 16 KB blocks of each half on their way out
constexpr uint32_t kACol = 256;      // the latents in TMEM, behind the two accumulators

struct ExpMisc {
  uint64_t afull;                    // latents of a slot tile
  uint64_t bfull[kBStages], bfree[kBStages];
  uint64_t dfull[2], dfree[2];       // accumulators
  uint64_t done;
  int tmp[35];
  alignas(16) int odd[2][4];         // first slot of a warp whose values are not all finite; by turns of units
  uint32_t tmem;
  int abort_flag;
};
constexpr uint32_t kExpSmem = 1024 + kBStages * kBBytes + 2 * kOutBufs * kBlk + sizeof(ExpMisc);
static_assert(kExpSmem <= 227 * 1024, "one block's shared memory");

// Slot tiles of a request, and one more than the workspace holds at most (so
// that sums over 320 requests fit 31 bits).
__device__ __forceinline__ int slot_tiles(const PrefillArgs& a, int q, bool report) {
  if (q >= a.Q) return 0;
  return min((prefill_chunk(a, q, report).end + kSlotTile - 1) / kSlotTile, (int)(a.cap / kSlotTile) + 1);
}

// The walk over units (slot tile, head), heads within a tile.
struct ExpWalk {
  int q, tile, h;   // request, its slot tile, head
  int tiles, end;   // the request's
  int64_t off;      // its first workspace row
  __device__ __forceinline__ void open(const PrefillArgs& a) {
    const Chunk c = prefill_chunk(a, q, false);
    end = c.end;
    tiles = (c.end + kSlotTile - 1) / kSlotTile;
  }
  __device__ __forceinline__ void step(const PrefillArgs& a) {
    if (++h < a.H) return;
    h = 0;
    ++tile;
    while (tile >= tiles) {  // (a caller that steps past the last unit does not look further)
      off += (int64_t)tiles * kSlotTile;
      tile = 0;
      if (++q >= a.Q) return;
      open(a);
    }
  }
};

__global__ void __launch_bounds__(kExpThreads, 1)
    k_expand_tc(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_kv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* b_sm = smem;
  uint8_t* o_sm = b_sm + kBStages * kBBytes;
  ExpMisc& ms = *reinterpret_cast<ExpMisc*>(o_sm + 2 * kOutBufs * kBlk);
  const uint32_t b_at = smem_u32(b_sm), o_at = smem_u32(o_sm);
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const Ctl ctl{&ms.abort_flag, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ms.abort_flag = 0;
    mbar_init(bar(ms.afull), 8);
    for (int i = 0; i < kBStages; ++i) {
      mbar_init(bar(ms.bfull[i]), 1);
      mbar_init(bar(ms.bfree[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ms.dfull[i]), 1);
      mbar_init(bar(ms.dfree[i]), 4);
    }
    mbar_init(bar(ms.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // (TMEM behind the wait for the kernel before, whichever that is, and ahead of
  // the release of the attention, which takes its own before it waits)
  pdl_wait();
  if (warp == 9) tmem_alloc(smem_u32(&ms.tmem), 512);

  // This block's units.  Requests in order; one that does not fit the
  // workspace ends the list (those behind it do not fit either).
  ExpWalk w{};
  int n_units = 0;
  {
    const bool report = blockIdx.x == 0 && (a.Q > 32 || warp == 0);
    const auto full = [&](int q, int t) { raise_error(a.err, ERR_CAPACITY, q, (uint32_t)t * kSlotTile); };
    const int cap_tiles = (int)(a.cap / kSlotTile);
    int u0 = 0;
    auto share = [&](int tiles) {  // the block's units; all fit 31 bits (the host's check)
      u0 = range_begin(tiles * a.H, gridDim.x, blockIdx.x);
      n_units = range_begin(tiles * a.H, gridDim.x, blockIdx.x + 1) - u0;
      return u0 / a.H;
    };
    int tiles_before = 0, want;
    if (a.Q <= 32) {
      // each warp by itself, a request a lane: no barriers
      const int t = slot_tiles(a, lane, report), upto = warp_inclusive_scan(t);
      if (report && t && upto > cap_tiles) full(lane, t);
      const uint32_t fits = __ballot_sync(0xffffffffu, upto <= cap_tiles);
      const int total = __shfl_sync(0xffffffffu, upto, fits ? 31 - __clz((int)fits) : 0);
      want = share(fits ? total : 0);
      const uint32_t here = __ballot_sync(0xffffffffu, upto - t <= want && want < upto);
      w.q = here ? __ffs((int)here) - 1 : 0;
      tiles_before = __shfl_sync(0xffffffffu, upto - t, w.q);
    } else {
      constexpr int kMany = 1 << 30;  // more tiles than any workspace has
      int total = 0, carry = 0;
      for (int base = 0; base < a.Q; base += kExpThreads) {
        const int q = base + (int)threadIdx.x, t = slot_tiles(a, q, report);
        int sum, kept;
        const int upto = carry + block_exclusive_scan(t, ms.tmp, &sum) + t;
        if (report && t && upto > cap_tiles) full(q, t);
        block_exclusive_scan(upto <= cap_tiles ? t : 0, ms.tmp, &kept);
        total += kept;
        carry = min(carry + sum, kMany);
      }
      want = share(total);
      carry = 0;
      for (int base = 0; base < a.Q && n_units; base += kExpThreads) {
        const int q = base + (int)threadIdx.x, t = slot_tiles(a, q, false);
        int sum;
        const int ex = carry + block_exclusive_scan(t, ms.tmp, &sum);
        if (ex <= want && want < ex + t) {
          ms.tmp[33] = q;
          ms.tmp[34] = ex;
        }
        carry = min(carry + sum, kMany);
        if (carry > want) break;
      }
      __syncthreads();
      if (n_units) {
        w.q = ms.tmp[33];
        tiles_before = ms.tmp[34];
      }
    }
    if (n_units) {
      w.off = (int64_t)tiles_before * kSlotTile;
      w.tile = want - tiles_before;
      w.h = u0 - want * a.H;
      w.open(a);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ms.tmem;
  pdl_release();

  if (!n_units) {
    // more blocks than units
  } else if (warp == 8) {
    // ======================= copies of the weights =======================
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    uint32_t armed[kBStages];
    for (int i = 0; i < kBStages; ++i) armed[i] = 2;
    for (int i = 0; i < n_units && ok; ++i) {
      for (int x = 0; x < 2 * kDC / kStageK; ++x) {
        const int k = x % (kDC / kStageK) * kStageK, row = w.h * kN + x / (kDC / kStageK) * kHalf;
        ok = wait_warp(bar(ms.bfree[st]), ph ^ 1u, ctl);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(bar(ms.bfull[st]), kBBytes);
          for (int c = 0; c < kStageK / 64; ++c)
            tma_load_2d(b_at + st * kBBytes + c * kBlk, &map_w, bar(ms.bfull[st]), k + c * 64, row);
        }
        armed[st] = ph;
        if (++st == kBStages) {
          st = 0;
          ph ^= 1u;
        }
      }
      w.step(a);
    }
    if (lane == 0 && ms.abort_flag)
      for (int s = 0; s < kBStages; ++s)
        if (armed[s] < 2) drain(bar(ms.bfull[s]), armed[s]);
  } else if (warp == 9) {
    // ======================= MMA issue =======================
    const uint32_t id = idesc_bf16(128, kHalf, 0, 0);
    int st = 0, nload = -1, seen = -1, q_seen = -1;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < n_units && ok; ++i) {
      if (w.tile != seen || w.q != q_seen) {
        seen = w.tile;
        q_seen = w.q;
        ++nload;
        ok = wait_warp(bar(ms.afull), (uint32_t)nload & 1u, ctl);
      }
      for (int half = 0; half < 2 && ok; ++half) {
        const uint32_t d = tmem + (uint32_t)half * kHalf;
        ok = wait_warp(bar(ms.dfree[half]), (uint32_t)i & 1u ^ 1u, ctl);
        for (int x = 0; x < kDC / kStageK && ok; ++x) {
          ok = wait_warp(bar(ms.bfull[st]), ph, ctl);
          if (!ok) break;
          fence_after();
          const uint64_t bd = sw128_desc(b_at + st * kBBytes, 16, 1024);
          const uint32_t at = tmem + kACol + (uint32_t)x * (kStageK / 2);
          const uint32_t joined = x > 0;
          if (elect()) {
#pragma unroll
            for (int kk = 0; kk < kStageK / 16; ++kk)
              mma_f16_ts(d, at + kk * 8, bd + (kk >> 2) * (kBlk >> 4) + 2 * (kk & 3), id, kk > 0 ? 1u : joined);
            commit(bar(ms.bfree[st]));
            if (x == kDC / kStageK - 1) commit(bar(ms.dfull[half]));
          }
          __syncwarp();
          if (++st == kBStages) {
            st = 0;
            ph ^= 1u;
          }
        }
      }
      w.step(a);
    }
    if (elect()) commit(bar(ms.done));
    __syncwarp();
    drain(bar(ms.done), 0);
  } else {
    // ======================= latents and epilogue =======================
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const LatentCache& C = a.cache;
    // A slot tile's latents: a thread's slot into its TMEM lane, two elements a
    // column.  Slots past the request's last become zeros, and so do their keys
    // and values.  The rotary part goes straight to the workspace.
    // Each half of the warps takes four of the eight 64-column pieces.
    // A warp brings its 32 slots' pieces by way of shared memory (the output
    // buffers' place), eight lanes a 128-byte line, 64 columns at a time and one
    // step ahead; the lines are asked into L2 all at once before (for the next
    // tile while this one's products run).  Each thread reading its own slot's
    // row took 10 us a tile, four units' time.
    auto place = [&](const ExpWalk& w, bool report) -> const uint4* {
      const int slot = w.tile * kSlotTile + row;
      if (slot >= w.end) return nullptr;
      const int page = C.bt[(int64_t)w.q * C.bt_stride + (slot >> C.log2b)];
      if (page < 0 || page >= C.num_pages) {
        if (report) raise_error(a.err, ERR_PAGE, w.q, (uint32_t)page);
        return nullptr;
      }
      return reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(C.data) +
                                            (((int64_t)page << C.log2b) + (slot & (C.b - 1))) * (kDC + kDR));
    };
    auto ask = [&](const uint4* src) {
      if (!src) return;
#pragma unroll
      for (int c = 0; c < (kDC + kDR) / 64; ++c)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 8 * c) : "memory");
    };
    auto load = [&](const ExpWalk& w) {
      const int slot = w.tile * kSlotTile + row;
      const uint4* src = place(w, true);
      ask(src);
      // this lane's piece of rows lane / 8 + 4 j
      const char* from[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        from[j] = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, (unsigned long long)src, (lane >> 3) + 4 * j));
      const uint32_t stage = o_at + (half * kOutBufs) * kBlk + (warp & 3) * 4096;
      auto fetch = [&](int c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int to = (lane >> 3) + 4 * j;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           stage + (c & 1) * kBlk + to * 128 + (((lane & 7) ^ (to & 7)) << 4)),
                       "l"(from[j] ? from[j] + c * 128 + (lane & 7) * 16 : reinterpret_cast<const char*>(C.data)),
                       "r"(from[j] ? 16u : 0u)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      constexpr int kPieces = kDC / 64 / 2;
      fetch(half * kPieces);
#pragma unroll 1
      for (int c = half * kPieces; c < (half + 1) * kPieces; ++c) {
        if (c + 1 < (half + 1) * kPieces) {
          fetch(c + 1);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        uint32_t v[32];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[4 * k]), "=r"(v[4 * k + 1]), "=r"(v[4 * k + 2]), "=r"(v[4 * k + 3])
                       : "r"(stage + (c & 1) * kBlk + lane * 128 + ((k ^ (lane & 7)) << 4))
                       : "memory");
        tmem_st32(tmem + lanes + kACol + (uint32_t)c * 32, v);
        __syncwarp();  // the buffer has been read
      }
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms.afull));
      if (half && w.h == 0) {  // (a tile that another block begins has its rotary part from there)
        char* dst = reinterpret_cast<char*>(a.kr) + (w.off + slot - lane + (lane >> 3)) * (kDR * 2) + (lane & 7) * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(dst + j * (4 * kDR * 2)) =
              from[j] ? *reinterpret_cast<const uint4*>(from[j] + kDC * 2 + (lane & 7) * 16) : make_uint4(0, 0, 0, 0);
      }
    };
    const bool store = (threadIdx.x & 127) == 0;  // the half's thread that issues its stores
    auto ask_behind = [&](ExpWalk at, int unit) {  // the tile behind that of `at`, the block's unit `unit`
      if (unit + a.H - at.h >= n_units) return;
      at.h = a.H - 1;
      at.step(a);
      ask(place(at, false));
    };
    // the next tile's latents, once every product of this one is complete
    auto reload = [&](const ExpWalk& next) {
      // (they pass through the stores' place)
      if (store) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      bar_sync(1 + half, 128);
      load(next);
    };
    int buf = 0;
    bool ok = true;
    load(w);
    if (half) ask_behind(w, 0);
    for (int i = 0; i < n_units; ++i) {
      ok = ok && wait_warp(bar(ms.dfull[half]), (uint32_t)i & 1u, ctl);
      if (bar_or(1 + half, 128, !ok)) break;  // (the warps leave together: they meet at barriers below)
      fence_after();
      ExpWalk next = w;
      if (i + 1 < n_units) next.step(a);
      const bool turn = next.tile != w.tile || next.q != w.q;
      if (half && turn) {  // before the epilogue, so that the next products begin
        reload(next);
        ask_behind(next, i + 1);
      }
      bool odd = false;  // of the values, not all are finite
#pragma unroll 1
      for (int c = 0; c < kHalf / 64; ++c) {
        uint32_t v[2][32];
        tmem_ld32(tmem + lanes + (uint32_t)(half * kHalf + c * 64), v[0]);
        tmem_ld32(tmem + lanes + (uint32_t)(half * kHalf + c * 64 + 32), v[1]);
        tmem_wait_ld();
        if (c == kHalf / 64 - 1) {  // the accumulator is in registers: hand it back
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(ms.dfree[half]));
        }
        uint32_t p[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
          p[k] = pack_bf16(__uint_as_float(v[k >> 4][2 * k & 31]), __uint_as_float(v[k >> 4][(2 * k & 31) + 1]));
        // Values that are not finite in bf16 are written as zeros: rows before the
        // slot, whose weights for it are 0, must not meet them.  Rows that attend to
        // the slot learn of it by the tile's first such slot.
        if (half) {
          uint32_t most = 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) most = __vmaxu2(most, p[k] & 0x7fff7fffu);
          const bool clear = (most & 0xffffu) >= 0x7f80u || most >> 16 >= 0x7f80u;
          if (clear)
#pragma unroll
            for (int k = 0; k < 32; ++k) p[k] = 0;
          odd |= clear;
          const uint32_t who = __ballot_sync(0xffffffffu, odd);
          if (lane == 0) ms.odd[i & 1][warp & 3] = who ? w.tile * kSlotTile + row + __ffs((int)who) - 1 : kNoSlot;
        }
        // the block's buffer: its store two blocks ago has read it
        if (store) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOutBufs - 1) : "memory");
        bar_sync(1 + half, 128);
        const uint32_t out = o_at + (half * kOutBufs + buf) * kBlk, dst = out + row * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((j ^ (row & 7)) << 4)), "r"(p[4 * j]),
                       "r"(p[4 * j + 1]), "r"(p[4 * j + 2]), "r"(p[4 * j + 3])
                       : "memory");
        fence_async_smem();
        bar_sync(1 + half, 128);
        if (store) {
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                           (uint64_t)&map_kv),
                       "r"(out), "r"(half * kHalf + c * 64), "r"((int)(w.h * a.cap + w.off + w.tile * kSlotTile))
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        buf ^= 1;
      }
      if (half && store) {
        const int4 first = *reinterpret_cast<const int4*>(ms.odd[i & 1]);
        a.odd[w.h * (a.cap / kSlotTile) + w.off / kSlotTile + w.tile] =
            min(min(first.x, first.y), min(first.z, first.w));
      }
      if (turn && !half) {
        // (of the keys' warps the epilogue comes first: the values' products run meanwhile)
        ok = wait_warp(bar(ms.dfull[1]), (uint32_t)i & 1u, ctl);
        if (bar_or(1 + half, 128, !ok)) break;
        reload(next);
      }
      w = next;
    }
    if (store) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kAttThreads = 352;  // warps 0..3 and 4..7 the two row tiles' softmax, 8 copies, 9 and 10 MMA issue
constexpr int kRing = 8;
constexpr int kKBlocks = 3, kVBlocks = 2, kKV = kKBlocks + kVBlocks;

// Which rows of which head a block takes.  A class is 256 rows of a request.
// The classes are ranked by their key tiles, longest first, and the units
// (class, head) go to the blocks in that order, so that what starts last is
// short.  The units behind the last full round of kTail blocks are cut along the
// keys into as many parts as fill the round, each part's maximum, sum and
// unnormalised output left in the workspace for the join (a chunk of few rows
// on a long context is cut into up to kMaxParts).  Against blocks in plain order: 1.15 -> 1.08
// ms (4096 rows on 16K slots x 32 heads), 134 -> 68 us (64 rows on 6000 slots x
// 16 heads).  The plan and the join cost some 5 us, so parts have kMinPart key
// tiles at least (with 4 instead of 8: 46.8 us, not 39.8, for 1000 rows x 4 heads), and
// where max_slots cannot give two such parts blocks go in plain order (35.6 us),
// as they do for more than kPlanClasses classes: each block ranks them, in time that
// grows with their square.
constexpr int kTail = 148, kMaxParts = 16, kPlanClasses = 256, kMinPart = 8;
struct Plan {
  int order[kPlanClasses];  // classes by rank; the empty ones last
  int tiles[kPlanClasses];  // key tiles by class
  int used;                 // classes that are not empty
};
struct Unit {
  int q, r0, h;
  int part, parts;
  int slot;  // of the parts in the workspace
};

// All threads of the block (a multiple of 32 threads).
__device__ __forceinline__ void make_plan(const PrefillArgs& a, Plan& p) {
  const int per = (a.rows + 2 * kRowTile - 1) / (2 * kRowTile), classes = a.Q * per;
  if (threadIdx.x == 0) p.used = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < classes; c += blockDim.x) {
    const int q = c / per, r0 = (c - q * per) * 2 * kRowTile;
    const Chunk ch = prefill_chunk(a, q, false);
    int64_t off = 0;
    for (int i = 0; i < q; ++i) off += (prefill_chunk(a, i, false).end + kSlotTile - 1) / kSlotTile * kSlotTile;
    const bool any = r0 < ch.count && off + ch.end <= a.cap;
    p.tiles[c] = any ? (ch.ctx - 2 + min(ch.count, r0 + 2 * kRowTile)) / kRowTile + 1 : 0;
    if (any) atomicAdd(&p.used, 1);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < classes; c += blockDim.x) {
    const int n = p.tiles[c];
    int rank = 0;
    for (int i = 0; i < classes; ++i) rank += p.tiles[i] > n || (p.tiles[i] == n && i < c);
    p.order[rank] = c;
  }
  __syncthreads();
}
// Unit u of the ranked ones.
__device__ __forceinline__ Unit unit_at(const PrefillArgs& a, const Plan& p, int u) {
  const int per = (a.rows + 2 * kRowTile - 1) / (2 * kRowTile);
  // one request: head by head, so that a head's keys are read by its rows at once
  const int c = p.order[a.Q == 1 ? u % p.used : u / a.H];
  return {c / per, c % per * 2 * kRowTile, a.Q == 1 ? u / p.used : u % a.H, 0, 1, 0};
}
// The tail's units, and the parts of one with n key tiles.
__device__ __forceinline__ int tail_of(const PrefillArgs& a, const Plan& p) { return p.used * a.H % kTail; }
__device__ __forceinline__ int parts_of(int tail, int n) {
  return max(1, min(min(kTail / tail, kMaxParts), n / kMinPart));
}

struct AttMisc {
  uint64_t kfull[2], vfull[2];  // K(i), V(i) landed: barrier i % 2 (the ring holds less than two key tiles)
  uint64_t empty[kRing];
  uint64_t qfull[2], sfull[2], pfull[2][2], odone[2];
  uint64_t olast[2];             // every second product of the row tile
  uint64_t turn[2];
  uint64_t done[2];
  int64_t tmp[33];
  uint32_t tmem;
  int abort_flag;
};
constexpr uint32_t kAttSmem = 1024 + 2 * kKBlocks * kBlk + kRing * kBlk + sizeof(AttMisc);
static_assert(kAttSmem <= 227 * 1024, "one block's shared memory");

__global__ void __launch_bounds__(kAttThreads, 1)
    k_prefill_tc(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_kr) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_sm = smem;
  uint8_t* r_sm = q_sm + 2 * kKBlocks * kBlk;
  AttMisc& ms = *reinterpret_cast<AttMisc*>(r_sm + kRing * kBlk);
  const uint32_t q_at = smem_u32(q_sm), r_at = smem_u32(r_sm);
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const Ctl ctl{&ms.abort_flag, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // What does not depend on the expanded keys runs while those are made: the
  // expansion has begun, so the lengths and the block table are there.  (A
  // block with nothing to do waits for it all the same: the launch must not
  // complete before it.)
  Unit w;
  if (a.planned) {
    Plan& p = *reinterpret_cast<Plan*>(r_sm);  // (the ring is not in use yet)
    make_plan(a, p);
    const int units = p.used * a.H, tail = tail_of(a, p), whole = units - tail;
    int u = blockIdx.x;
    if (u >= whole) {
      if (!tail) return pdl_enter();
      const int most = min(kTail / tail, kMaxParts), x = u - whole;
      u = whole + x / most;
      if (u >= units) return pdl_enter();
      w = unit_at(a, p, u);
      w.part = x % most;
      w.parts = parts_of(tail, p.tiles[p.order[a.Q == 1 ? u % p.used : u / a.H]]);
      w.slot = x;
      if (w.part >= w.parts) return pdl_enter();
    } else {
      w = unit_at(a, p, u);
    }
    fence_async_smem();  // the plan has been read; copies through the async proxy take its place
    __syncthreads();
  } else {
    const int per = (a.rows + 2 * kRowTile - 1) / (2 * kRowTile);
    const int c = blockIdx.x / a.H;
    w = {c / per, (per - 1 - c % per) * 2 * kRowTile, (int)blockIdx.x % a.H, 0, 1, 0};
  }
  const int h = w.h, q = w.q, r0 = w.r0;
  const Chunk ch = prefill_chunk(a, q, false);
  if (r0 >= ch.count) return pdl_enter();
  const int64_t off = prefill_rows_before(a, q, ms.tmp);
  if (off + ch.end > a.cap) return pdl_enter();
  {
    const LatentCache& C = a.cache;
    int bad = 0;
    for (int i = threadIdx.x; i <= (ch.end - 1) >> C.log2b; i += kAttThreads) {
      const int page = C.bt[(int64_t)q * C.bt_stride + i];
      bad |= page < 0 || page >= C.num_pages;
    }
    if (__syncthreads_or(bad)) return pdl_enter();
  }
  // rows and key tiles of the two row tiles
  const int rows0 = min(ch.count - r0, kRowTile), rows1 = max(0, min(ch.count - r0 - kRowTile, kRowTile));
  const int pos0 = ch.ctx - 1 + r0;  // of the first row
  const int all0 = (pos0 + rows0 - 1) / kRowTile + 1, all1 = rows1 ? (pos0 + kRowTile + rows1 - 1) / kRowTile + 1 : 0;
  // of these the block takes key tiles i0 .. i0 + n - 1, of which row tile t sees the first n0, n1
  const int all = max(all0, all1);
  const int i0 = all * w.part / w.parts, n = all * (w.part + 1) / w.parts - i0;
  const int n0 = max(0, min(all0 - i0, n)), n1 = max(0, min(all1 - i0, n));
  const bool two = rows1 > 0;

  if (threadIdx.x == 0) {
    ms.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) mbar_init(bar(ms.empty[i]), two ? 2 : 1);  // the row tiles' MMA warps
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(ms.kfull[t]), 1);
      mbar_init(bar(ms.vfull[t]), 1);
      mbar_init(bar(ms.done[t]), 1);
      mbar_init(bar(ms.qfull[t]), 128);
      mbar_init(bar(ms.sfull[t]), 1);
      mbar_init(bar(ms.pfull[t][0]), 4);
      mbar_init(bar(ms.pfull[t][1]), 4);
      mbar_init(bar(ms.turn[t]), 1);
      mbar_init(bar(ms.odone[t]), 1);
      mbar_init(bar(ms.olast[t]), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // (ahead of the wait: the kernel before is the expansion, which had all its TMEM when it let this one in)
  if (warp == 9) tmem_alloc(smem_u32(&ms.tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ms.tmem;
  constexpr uint32_t kOCol = 256;
  pdl_enter();

  if (warp == 8) {
    // ======================= copies =======================
    uint32_t armed[4] = {2, 2, 2, 2};  // kfull, vfull
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n && ok; ++i) {
      const int row = (int)(off + (int64_t)(i0 + i) * kRowTile);
      const uint32_t kf = bar(ms.kfull[i & 1]), vf = bar(ms.vfull[i & 1]), par = (uint32_t)(i >> 1) & 1u;
#pragma unroll 1
      for (int b = 0; b < kKV; ++b) {
        ok = wait_warp(bar(ms.empty[s]), ph ^ 1u, ctl);
        if (!ok) break;
        if (lane == 0) {
          if (b == 0) mbar_expect_tx(kf, kKBlocks * kBlk);
          if (b == kKBlocks) mbar_expect_tx(vf, kVBlocks * kBlk);
          if (b < 2) {
            tma_load_2d(r_at + s * kBlk, &map_k, kf, b * 64, (int)(h * a.cap) + row);
          } else if (b == 2) {
            tma_load_2d(r_at + s * kBlk, &map_kr, kf, 0, row);
          } else {
            const int y = (int)(h * a.cap) + row + (b - kKBlocks) * 64;
            tma_load_2d(r_at + s * kBlk, &map_v, vf, kDN, y);
            tma_load_2d(r_at + s * kBlk + kBlk / 2, &map_v, vf, kDN + 64, y);
          }
        }
        if (b == 0) armed[i & 1] = par;
        if (b == kKBlocks) armed[2 + (i & 1)] = par;
        if (++s == kRing) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // (a group that an abort cut short never completes: its wait ends by its limit)
    if (lane == 0 && ms.abort_flag)
      for (int i = 0; i < 2; ++i) {
        if (armed[i] < 2) drain(bar(ms.kfull[i]), armed[i]);
        if (armed[2 + i] < 2) drain(bar(ms.vfull[i]), armed[2 + i]);
      }
  } else if (warp > 8) {
    // ======================= MMA issue, a warp for each row tile =======================
    // The products of one tile need their order, those of the two tiles do not;
    // while one warp waits (75 cycles even where all is there) the other's
    // instructions run.
    const int t = warp - 9, nt = t ? n1 : n0;
    const uint32_t id_s = idesc_bf16(128, 128, 0, 0);
    const uint32_t id_o = idesc_bf16(128, 128, 0, 1);
    const uint32_t s_col = tmem + t * 128, o_col = tmem + kOCol + t * 128;
    const uint64_t ad = sw128_desc(q_at + t * kKBlocks * kBlk, 16, 1024);
    // The elected lane's parts.  S(i): columns b of K, at ring block s.
    auto first = [&](int b, int s) {
      const uint64_t aq = ad + (uint64_t)b * (kBlk >> 4), bd = sw128_desc(r_at + s * kBlk, 16, 1024);
      const uint32_t joined = b > 0;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_f16(s_col, aq + 2 * kk, bd + 2 * kk, id_s, kk > 0 ? 1u : joined);
      commit(bar(ms.empty[s]));
    };
    // O += P V of half a key tile, V at ring block s.
    auto second = [&](int half, int s, uint32_t joined) {
      const uint64_t bd = sw128_desc(r_at + s * kBlk, kBlk / 2, 1024);
      const uint32_t p = s_col + half * 64;
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_f16_ts(o_col, p + k * 8, bd + k * (2048 >> 4), id_o, k > 0 ? 1u : joined);
      commit(bar(ms.empty[s]));
      commit(bar(ms.odone[t]));
    };
    bool ok = true;
    if (nt) {
      ok = wait_warp(bar(ms.qfull[t]), 0, ctl);
      // Turn i: the second product of key tile i, the first of i + 1 (turn -1: the first alone).  The tiles take
      // turns, so that one's softmax falls under the other's products (left to themselves they run in step).
      for (int i = -1; ok && i < nt; ++i) {
        if (i >= 0) {
          const int s = kKV * i + kKBlocks;
          ok = wait_warp(bar(ms.vfull[i & 1]), (uint32_t)(i >> 1) & 1u, ctl) &&
               wait_warp(bar(ms.pfull[t][0]), (uint32_t)i & 1u, ctl);
          if (ok && two && (t ? i < n0 : i > 0))
            ok = wait_warp(bar(ms.turn[t]), (uint32_t)(t ? i : i - 1) & 1u, ctl);
#pragma unroll 1
          for (int half = 0; ok && half < 2; ++half) {
            if (half) ok = wait_warp(bar(ms.pfull[t][1]), (uint32_t)i & 1u, ctl);
            if (!ok) break;
            fence_after();
            if (elect()) second(half, (s + half) % kRing, half || i > 0 ? 1u : 0u);
            __syncwarp();
          }
          if (!ok) break;
          if (i == nt - 1 && elect()) commit(bar(ms.olast[t]));
          __syncwarp();
        }
        if (i + 1 < nt) {
          ok = wait_warp(bar(ms.kfull[(i + 1) & 1]), (uint32_t)((i + 1) >> 1) & 1u, ctl);
          if (!ok) break;
          fence_after();
#pragma unroll 1
          for (int b = 0; b < kKBlocks; ++b) {
            // (the turn goes on before its last instructions)
            if (b == kKBlocks - 1 && two && i >= 0 && lane == 0) mbar_arrive(bar(ms.turn[t ^ 1]));
            if (elect()) first(b, (kKV * (i + 1) + b) % kRing);
            __syncwarp();
          }
          if (elect()) commit(bar(ms.sfull[t]));
          __syncwarp();
        } else if (two && lane == 0) {
          mbar_arrive(bar(ms.turn[t ^ 1]));
        }
      }
    }
    // The blocks of key tiles that only the other row tile sees: handed back
    // once they have landed, so that no block is handed back twice in one round
    // of the ring.
    if (t == 0 || two)
      for (int i = nt; ok && i < n; ++i) {
        ok = wait_warp(bar(ms.kfull[i & 1]), (uint32_t)(i >> 1) & 1u, ctl) &&
             wait_warp(bar(ms.vfull[i & 1]), (uint32_t)(i >> 1) & 1u, ctl);
        if (ok && lane < kKV) mbar_arrive(bar(ms.empty[(kKV * i + lane) % kRing]));
      }
    if (elect()) commit(bar(ms.done[t]));
    __syncwarp();
    drain(bar(ms.done[t]), 0);
  } else {
    // ======================= softmax and output =======================
    const int t = warp >> 2, tid = threadIdx.x & 127;
    const int nt = t ? n1 : n0, rows = t ? rows1 : rows0;
    const int64_t token0 = (int64_t)q * a.rows + r0 + t * kRowTile;
    if (nt) {
      // the tile's queries: 8 lanes a 128-byte line, rows behind the last as zeros
      const int piece = tid & 7;
#pragma unroll 1
      for (int row = tid >> 3; row < kRowTile; row += 16) {
        const bool live = row < rows;
        const char* src = reinterpret_cast<const char*>(a.q) +
                          ((live ? (token0 + row) * a.q_tok : 0) + h * a.q_head) * 2 + piece * 16;
        const uint32_t dst = q_at + t * kKBlocks * kBlk + row * 128 + ((piece ^ (row & 7)) << 4);
        if (a.q_vec) {
#pragma unroll
          for (int b = 0; b < kKBlocks; ++b)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + b * kBlk), "l"(src + b * 128),
                         "r"(live ? 16u : 0u)
                         : "memory");
        } else {
#pragma unroll 1
          for (int b = 0; b < kKBlocks; ++b) {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(src + b * 128);
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = live ? (uint32_t)e[2 * k] | (uint32_t)e[2 * k + 1] << 16 : 0u;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + b * kBlk), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3])
                         : "memory");
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      mbar_arrive(bar(ms.qfull[t]));
    }
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + kOCol + t * 128;
    const int pos = pos0 + t * kRowTile + tid - i0 * kRowTile;  // this thread's row, from the part's first key
    const int whole = (pos0 + t * kRowTile + 1) / 64 - 2 * i0;  // halves that every row of the tile sees whole
    const float scale = a.scale_log2;
    const float lazy = kLazy / scale;  // (infinite where no score can grow so far)
    float M = -INFINITY, l = 0.f;      // the reference, a score
    float limit = -INFINITY, ref = 0.f;  // the score that moves it, and M * scale (0 where M is far or nothing is seen)
    bool far = false, any_far = false;  // this row's M is far, one of the warp's rows'
    bool ok = true;
    // The first slot whose values are not finite (they are stored as zeros): a row that sees it becomes NaN.
    const int32_t* odd = a.odd + h * (a.cap / kSlotTile) + off / kSlotTile + i0;
    int spoilt = kNoSlot, first_odd = kNoSlot;
    // halves of 64 keys
    for (int j = 0; j < 2 * nt; ++j) {
      const uint32_t at = s_at + (j & 1) * 64;
      if (!(j & 1)) first_odd = odd[j >> 1];
      // (S of a key tile follows the second products of the tile before)
      if (!(j & 1)) ok = wait_warp(bar(ms.sfull[t]), (uint32_t)(j >> 1) & 1u, ctl);
      if (!ok) break;
      fence_after();
      uint32_t s[2][32];
      tmem_ld32(at, s[0]);
      tmem_ld32(at + 32, s[1]);
      tmem_wait_ld();
      if (j >= whole) {
        const int left = pos - j * 64;  // columns 0 .. left are seen
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c > left) s[c >> 5][c & 31] = 0xff800000u;
      }
      float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 32; c += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mt[k] = max3(mt[k], __uint_as_float(s[0][c + k]), __uint_as_float(s[1][c + k]));
      const float top = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
      // (at the first half M is -inf; a row's reference moves by its own maximum alone, so that its bits do not
      // depend on what its warp's other rows see)
      const bool grown = top > limit;
      if (__any_sync(0xffffffffu, grown)) {
        const float f = grown ? moved(M, top, scale) : 1.f;
        if (grown) {
          M = top;
          limit = M + lazy;
          ref = M * scale;
          far = fabsf(ref) >= kFar;
          if (far) ref = 0.f;
        }
        any_far = __any_sync(0xffffffffu, far);
        l *= f;
        if (j > 0) {
          // (of the second products only the last can still be running: S, or the half before, waited for the others)
          ok = wait_warp(bar(ms.odone[t]), (uint32_t)(j - 1) & 1u, ctl);
          if (!ok) break;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(o_at + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(o_at + c * 16, o);
          }
        }
      }
      if (any_far) {
        // the scores less M, by way of their place in TMEM (64 subtractions here would cost every row)
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t x[16];
          tmem_ld16(at + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            x[k] = c + k > pos - j * 64 ? 0xff800000u : __float_as_uint(__uint_as_float(x[k]) - (far ? M : 0.f));
          tmem_st16(at + c, x);
        }
        tmem_wait_st();
        tmem_ld32(at, s[0]);
        tmem_ld32(at + 32, s[1]);
        tmem_wait_ld();
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t p[32];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        // four weights: two packed multiply-adds, two packed sums
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const int e = 2 * c + k;
          fma2(x[k], x[k + 1], __uint_as_float(s[e >> 5][e & 31]), __uint_as_float(s[e >> 5][(e & 31) + 1]), scale,
               -ref);
          x[k] = ex2(x[k]);
          x[k + 1] = ex2(x[k + 1]);
          add2(sum[k], sum[k + 1], x[k], x[k + 1]);
          p[c + k / 2] = pack_bf16(x[k], x[k + 1]);
        }
      }
      tmem_st32(at, p);
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ms.pfull[t][j & 1]));
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      spoilt = min(spoilt, first_odd);
    }
    if (spoilt <= pos0 + t * kRowTile + tid) l = __int_as_float(0x7fffffff);
    // (a barrier of one phase: the products behind this warp's last weights may be complete before it looks, and
    // odone's parity would not tell)
    if (ok && nt) ok = wait_warp(bar(ms.olast[t]), 0, ctl);
    if (ok && w.parts > 1) {
      // a part: unnormalised, for the join
      const int64_t at = (int64_t)w.slot * 2 * kRowTile + t * kRowTile + tid;
      if (tid < rows) a.part_ml[at] = make_float2(M * scale, l);
      if (nt) {
        fence_after();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(o_at + c * 16, o);
          tmem_wait_ld();
          if (tid < rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(a.part + at * kDV + c * 16 + 4 * k) =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
    } else if (ok && nt) {
      fence_after();
      const float norm = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + ((token0 + tid) * a.H + h) * kDV;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(o_at + c * 32, o);
        tmem_wait_ld();
        if (tid < rows) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = pack_bf16(__uint_as_float(o[8 * k + 2 * e]) * norm, __uint_as_float(o[8 * k + 2 * e + 1]) * norm);
            *reinterpret_cast<uint4*>(out + c * 32 + k * 8) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the parts of the tail's units: a warp a row at a time, in part order.
// Bound by the parts' bytes (19 MB at most) out of L2 and HBM: 5 to 20 us.
// grid (units, kJoinGroups groups of rows); few blocks, since each makes the plan.
constexpr int kJoinGroups = 4;
__global__ void __launch_bounds__(256) k_prefill_join(const __grid_constant__ PrefillArgs a) {
  __shared__ Plan p;
  make_plan(a, p);  // (the lengths were there before the attention started)
  pdl_enter();
  const int tail = tail_of(a, p), x = blockIdx.x;
  if (x >= tail) return;
  const int u = p.used * a.H - tail + x;
  const Unit w = unit_at(a, p, u);
  const int most = min(kTail / tail, kMaxParts);
  const int parts = parts_of(tail, p.tiles[p.order[a.Q == 1 ? u % p.used : u / a.H]]);
  if (parts == 1) return;
  const Chunk ch = prefill_chunk(a, w.q, false);
  const int lane = threadIdx.x & 31;
  {
    const LatentCache& C = a.cache;
    int bad = 0;
    for (int i = threadIdx.x; i <= (ch.end - 1) >> C.log2b; i += 256) {
      const int page = C.bt[(int64_t)w.q * C.bt_stride + i];
      bad |= page < 0 || page >= C.num_pages;
    }
    if (__syncthreads_or(bad)) return;
  }
  const int64_t at0 = (int64_t)x * most * 2 * kRowTile;
  const int rows = min(2 * kRowTile, ch.count - w.r0);
  for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < rows; row += kJoinGroups * 8) {
    const float2 ml = lane < parts ? a.part_ml[at0 + (int64_t)lane * 2 * kRowTile + row] : make_float2(-INFINITY, 0.f);
    float m = ml.x;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float wt = m == -INFINITY ? 0.f : exp2f(ml.x - m);
    float l = ml.y * wt;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
      const float4 v = wi != 0.f ? *reinterpret_cast<const float4*>(
                                       a.part + (at0 + (int64_t)i * 2 * kRowTile + row) * kDV + 4 * lane)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
      o.x = fmaf(wi, v.x, o.x);
      o.y = fmaf(wi, v.y, o.y);
      o.z = fmaf(wi, v.z, o.z);
      o.w = fmaf(wi, v.w, o.w);
    }
    const float norm = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint2 v;
    v.x = pack_bf16(o.x * norm, o.y * norm);
    v.y = pack_bf16(o.z * norm, o.w * norm);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                              (((int64_t)w.q * a.rows + w.r0 + row) * a.H + w.h) * kDV + 4 * lane) = v;
  }
}

}  // namespace

// bf16 at the widths these kernels are made for, with 16-byte alignment; all else takes the CUDA-core kernels.
bool prefill_tc_supported(const PrefillArgs& a, int bf16) {
  // workspace rows are the tensor maps' 32-bit coordinates; units fit 31 bits
  return bf16 && a.cache.dc == kDC && a.cache.dr == kDR && a.dn == kDN && a.dv == kDV &&
         ((uintptr_t)a.cache.data & 15) == 0 && ((uintptr_t)a.w & 15) == 0 && ((uintptr_t)a.out & 15) == 0 &&
         ((int64_t)a.cache.num_pages << a.cache.log2b) < (int64_t(1) << 31) &&
         a.cap * a.H < (int64_t(1) << 31);
}

cudaError_t prepare_prefill_tc() {
  const cudaError_t e = cudaFuncSetAttribute(k_expand_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kExpSmem);
  return e == cudaSuccess
             ? cudaFuncSetAttribute(k_prefill_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAttSmem)
             : e;
}

cudaError_t launch_prefill_tc(const PrefillArgs& a, void* encode_fn, int sms, cudaStream_t s) {
  CUtensorMap mw, mkv, mv, mkr;
  if (!encode_rows(encode_fn, &mw, a.w, (uint64_t)a.H * kN, kDC, kDC * 2, kHalf) ||
      !encode_rows(encode_fn, &mkv, a.kv, (uint64_t)a.H * a.cap, kN, kN * 2, kRowTile) ||
      !encode_rows(encode_fn, &mv, a.kv, (uint64_t)a.H * a.cap, kN, kN * 2, kRowTile / 2) ||
      !encode_rows(encode_fn, &mkr, a.kr, (uint64_t)a.cap, kDR, kDR * 2, kRowTile))
    return cudaErrorInvalidValue;
  cudaError_t e;
  {
    PdlLaunch l(dim3((unsigned)sms), dim3(kExpThreads), kExpSmem, s);
    e = cudaLaunchKernelEx(&l.cfg, k_expand_tc, a, mw, mkv);
  }
  if (e != cudaSuccess) return e;
  const int64_t classes = (int64_t)a.Q * ((a.rows + 2 * kRowTile - 1) / (2 * kRowTile));
  PrefillArgs b = a;
  b.planned = classes <= kPlanClasses && (a.max_slots + kRowTile - 1) / kRowTile >= 2 * kMinPart;
  {
    PdlLaunch l(dim3((unsigned)(classes * a.H + (b.planned ? kTail : 0))), dim3(kAttThreads), kAttSmem, s);
    e = cudaLaunchKernelEx(&l.cfg, k_prefill_tc, b, mkv, mv, mkr);
  }
  if (e != cudaSuccess || !b.planned) return e;
  PdlLaunch l(dim3((unsigned)std::min<int64_t>(kTail - 1, classes * a.H), kJoinGroups), dim3(256), 0, s);
  return cudaLaunchKernelEx(&l.cfg, k_prefill_join, b);
}

}  // namespace spin
